// New tokens into the paged pool: the per-head RMS norm of queries and keys, their rotation to
// the tokens' positions and the write of K and V to the tokens' slots, in one pass.
//
//   GQA: q' = R(p) (q * rsqrt(mean q^2 + eps) * w_q) per query head, k' likewise with w_k into
//        the K row, v copied into the V row.
//   MLA: the latent c_KV normed with w_k and the k_pe band rotated into the row; the queries
//        (absorbed form) keep their latent part and turn their rope band.
//
// One CTA of 256 threads per kTok tokens. It first builds the tokens' phase table (each (token,
// pair) once, by the exact Q0.64 range reduction of the other kernels; every head of the token
// reads it) and resolves their slots. Then W = 2^ceil(log2(band / 16)) lanes take one (token,
// head) item: a lane holds the two 8-column chunks of a column unit, which are closed under
// pairing, so the norm is one shuffle reduction over the W lanes and the rotation needs no
// exchange. Sums of squares, the norm and the rotation are float32; each output is rounded to
// bf16 once.
// Bound: HBM (every byte is read and written once) at many tokens, latency at few.
#include "kamera_dev.cuh"

namespace kamera {

namespace {

constexpr int kThr = 256;
constexpr int kBatch = 4;  // items a group of lanes has in flight

__device__ __forceinline__ float sum_sq8(const float *x) {
  float s = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) s = fmaf(x[e], x[e], s);
  return s;
}

// The factor by which a row is scaled before its squares are summed: the sum of squares of bf16
// values can pass float32's range at either end, and a row whose mean square (with eps) lies
// near them is summed again, scaled by a power of two that brings it back. A NaN stays with 1.
__device__ __forceinline__ float norm_scale(float mean) {
  return mean > 0x1p126f ? 0x1p-70f : (mean < 0x1p-90f ? 0x1p70f : 1.f);
}

__device__ __forceinline__ uint4 ld16(const __nv_bfloat16 *p) {
  return *reinterpret_cast<const uint4 *>(p);  // plain: q_out may be q
}
__device__ __forceinline__ void st16(__nv_bfloat16 *p, const uint4 &v) {
  *reinterpret_cast<uint4 *>(p) = v;
}

template <int kTok>
__global__ void __launch_bounds__(kThr) append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ float2 cs[kTok * kMaxPairs];
  __shared__ long long slots[kTok];  // -1: no slot, K and V are not written
  __shared__ int live[kTok];         // 0: padding or a bad token, nothing is written
  const DevLayout &lay = a.lay;
  const int tid = threadIdx.x;
  const long long t0 = (long long)blockIdx.x * kTok;
  const int nt = (int)min((long long)kTok, a.T - t0);
  const int np = lay.npairs;
  for (int e = tid; e < nt * np; e += kThr) {
    const int t = e / np, i = e - t * np;
    const int axis = lay.mrope ? mrope_axis(lay, i) : 0;
    const int stride = lay.mrope ? 3 : 1;
    cs[e] = rope_phase(a.freq.q[i], __ldg(a.positions + (t0 + t) * stride + axis));
  }
  if (tid < nt) {
    const int req = __ldg(a.req + t0 + tid), tok = __ldg(a.tok + t0 + tid);
    const bool padding = req < 0;
    const bool bad = !padding && (req >= a.pool.num_reqs || tok < 0 ||
                                  tok >= (long long)a.pool.pt_stride * lay.page_size);
    if (bad) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
    live[tid] = !padding && !bad;
    slots[tid] = padding || bad ? -1 : slot_of(a.pool, lay.page_size, req, tok, a.status);
  }
  __syncthreads();

  const bool gqa = lay.kind == KAMERA_GQA;
  const long long layer_k = (long long)a.layer * a.pool.num_slots * lay.row_k;
  // rotated items: the query heads, then the key bands, of each token
  const int band = lay.rope_d, units = band >> 4;
  int w = 1;
  while (w < units) w <<= 1;
  const int sub = tid / w, q = tid & (w - 1), nsub = kThr / w;
  const int n_k = gqa ? lay.H : 1;
  const int per_tok = a.hq + n_k, items = per_tok * nt;
  const bool neox = lay.style == KAMERA_ROPE_NEOX_HALF;
  const int ca = neox ? 8 * q : 16 * q, cb = neox ? ca + (band >> 1) : ca + 8;
  const bool mine = q < units;
  for (int it0 = sub; it0 < items + sub; it0 += nsub * kBatch) {  // whole warps iterate alike
    uint4 ra[kBatch], rb[kBatch];
    __nv_bfloat16 *dst[kBatch];
    int tk[kBatch];
    bool isq[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int it = it0 + j * nsub;
      dst[j] = nullptr;
      tk[j] = 0;
      isq[j] = false;
      ra[j] = rb[j] = make_uint4(0, 0, 0, 0);
      if (it >= items || !mine) continue;
      const int t = it / per_tok, h = it - t * per_tok;
      tk[j] = t;
      const __nv_bfloat16 *src;
      if (h < a.hq) {
        if (!live[t]) continue;
        isq[j] = true;
        const int off = gqa ? h * lay.hd : h * lay.row_k + lay.latent;
        src = a.q + (t0 + t) * a.q_stride + off;
        dst[j] = a.q_out + (t0 + t) * a.q_out_stride + off;
      } else {
        if (slots[t] < 0) continue;
        const int off = gqa ? (h - a.hq) * lay.hd : lay.latent;
        src = a.k + (t0 + t) * a.k_stride + off;
        dst[j] = a.pool.k + layer_k + slots[t] * lay.row_k + off;
      }
      ra[j] = ld16(src + ca);
      rb[j] = ld16(src + cb);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      float xa[8], xb[8];
      unpack8(ra[j], xa);
      unpack8(rb[j], xb);
      const __nv_bfloat16 *wt = gqa ? (isq[j] ? a.q_weight : a.k_weight) : nullptr;
      if (gqa && (a.q_weight || a.k_weight)) {  // every lane takes part in the reduction
        auto mean_sq = [&]() {
          float s = sum_sq8(xa) + sum_sq8(xb);
          for (int o = w >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          return s / (float)band;
        };
        float mean = mean_sq() + a.eps;
        const float f = wt ? norm_scale(mean) : 1.f;
        if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            xa[e] *= f;
            xb[e] *= f;
          }
          mean = mean_sq() + a.eps * f * f;
        }
        if (wt && mine) {
          const float r = rsqrtf(mean);
          float wa[8], wb[8];
          unpack8(__ldg(reinterpret_cast<const uint4 *>(wt + ca)), wa);
          unpack8(__ldg(reinterpret_cast<const uint4 *>(wt + cb)), wb);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            xa[e] = xa[e] * r * wa[e];
            xb[e] = xb[e] * r * wb[e];
          }
        }
      }
      if (!dst[j]) continue;
      const float2 *c = cs + tk[j] * np;
      if (neox) {
#pragma unroll
        for (int e = 0; e < 8; ++e) rot_pair(xa[e], xb[e], c[8 * q + e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          rot_pair(xa[e], xa[e + 1], c[8 * q + (e >> 1)]);
          rot_pair(xb[e], xb[e + 1], c[8 * q + 4 + (e >> 1)]);
        }
      }
      st16(dst[j] + ca, pack8_rn(xa));
      st16(dst[j] + cb, pack8_rn(xb));
    }
  }

  if (gqa) {  // V rows, byte for byte
    const int nc = lay.row_v >> 3;
    __nv_bfloat16 *pv = a.pool.v + (long long)a.layer * a.pool.num_slots * lay.row_v;
    for (int e = tid; e < nt * nc; e += kThr) {
      const int t = e / nc, c = e - t * nc;
      if (slots[t] >= 0)
        st16(pv + slots[t] * lay.row_v + 8 * c, ld16(a.v + (t0 + t) * a.v_stride + 8 * c));
    }
    return;
  }
  // MLA: the queries' latent parts, byte for byte
  const int nc = lay.latent >> 3;
  if (a.q_out != a.q || a.q_out_stride != a.q_stride) {
    for (int e = tid; e < nt * a.hq * nc; e += kThr) {
      const int t = e / (a.hq * nc), r = e - t * (a.hq * nc), h = r / nc, c = r - h * nc;
      if (live[t])
        st16(a.q_out + (t0 + t) * a.q_out_stride + h * lay.row_k + 8 * c,
             ld16(a.q + (t0 + t) * a.q_stride + h * lay.row_k + 8 * c));
    }
  }
  // and the latent row, a warp to a token
  const int lane = tid & 31;
  for (int t = tid >> 5; t < nt; t += kThr / 32) {
    if (slots[t] < 0) continue;
    const __nv_bfloat16 *src = a.k + (t0 + t) * a.k_stride;
    __nv_bfloat16 *dst = a.pool.k + layer_k + slots[t] * lay.row_k;
    float r = 1.f, f = 1.f;
    if (a.k_weight) {
      auto mean_sq = [&]() {
        float s = 0.f;
        for (int c = lane; c < nc; c += 32) {
          float x[8];
          unpack8(ld16(src + 8 * c), x);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] *= f;
          s += sum_sq8(x);
        }
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        return s / (float)lay.latent;
      };
      float mean = mean_sq() + a.eps;
      f = norm_scale(mean);
      if (f != 1.f) mean = mean_sq() + a.eps * f * f;
      r = rsqrtf(mean);
    }
    for (int c = lane; c < nc; c += 32) {
      uint4 v = ld16(src + 8 * c);
      if (a.k_weight) {
        float x[8], wv[8];
        unpack8(v, x);
        unpack8(__ldg(reinterpret_cast<const uint4 *>(a.k_weight + 8 * c)), wv);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * f * r * wv[e];
        v = pack8_rn(x);
      }
      st16(dst + 8 * c, v);
    }
  }
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, cudaStream_t s) {
  append_kernel<1><<<(unsigned)a.T, kThr, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kamera
