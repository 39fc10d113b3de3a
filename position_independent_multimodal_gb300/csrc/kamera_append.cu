// New tokens into the paged pool: the per-head RMS norm of queries and keys, their rotation to
// the tokens' positions and the write of K and V to the tokens' slots, in one pass.
//
//   GQA: q' = R(p) (q * rsqrt(mean q^2 + eps) * w_q) per query head, k' likewise with w_k into
//        the K row, v copied into the V row.
//   MLA: the latent c_KV normed with w_k and the k_pe band rotated into the row; the queries
//        (absorbed form) keep their latent part and turn their rope band.
//
// One CTA of 256 threads per kTok tokens. W = 2^ceil(log2(band / 16)) lanes take one (token, head)
// item: a lane holds the two 8-column chunks of a column unit, which are closed under pairing, so
// the norm is one shuffle reduction over the W lanes and the rotation needs no exchange. A group
// of W lanes stays with one token and takes several of its heads at a time, so that their loads
// are in flight together, before the phases and slots are known, and its phases are read once.
// The CTA computes the tokens' phases (each (token, pair) once, by the exact Q0.64 range reduction
// of the other kernels) and resolves their slots while the first loads run. Sums of squares, the
// norm and the rotation are float32; each output is rounded to bf16 once.
// Bound: HBM (every byte is read and written once) at many tokens, latency at few.
#include "kamera_dev.cuh"

namespace kamera {

namespace {

constexpr int kThr = 256;
constexpr int kBatch = 4;  // items a group of lanes (rows a warp) has in flight

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
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long t0 = (long long)blockIdx.x * kTok;
  const int nt = (int)min((long long)kTok, a.T - t0);
  const int np = lay.npairs;
  const bool gqa = lay.kind == KAMERA_GQA;

  // rotated items: the query heads, then the key bands, of this group's token
  const int band = lay.rope_d, units = band >> 4;
  int w = 1;
  while (w < units) w <<= 1;
  const int q = tid & (w - 1), groups = kThr / w / kTok;  // groups of lanes per token
  const int sub = tid / w, tk = sub / groups, h_first = sub - tk * groups;
  const int per_tok = a.hq + (gqa ? lay.H : 1);
  const bool neox = lay.style == KAMERA_ROPE_NEOX_HALF;
  const int ca = neox ? 8 * q : 16 * q, cb = neox ? ca + (band >> 1) : ca + 8;
  const bool mine = q < units && tk < nt;
  const long long tok = t0 + tk;
  // column of head h in the queries' or keys' row
  auto column = [&](int h) {
    return gqa ? (h < a.hq ? h : h - a.hq) * lay.hd : (h < a.hq ? h * lay.row_k : 0) + lay.latent;
  };
  uint4 ra[kBatch], rb[kBatch];
  auto load = [&](int h0) {
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = h0 + j * groups;
      ra[j] = rb[j] = make_uint4(0, 0, 0, 0);
      if (mine && h < per_tok) {
        const __nv_bfloat16 *src =
            (h < a.hq ? a.q + tok * a.q_stride : a.k + tok * a.k_stride) + column(h);
        ra[j] = ld16(src + ca);
        rb[j] = ld16(src + cb);
      }
    }
  };
  load(h_first);

  for (int e = tid; e < nt * np; e += kThr) {
    const int t = e / np, i = e - t * np;
    const int axis = lay.mrope ? mrope_axis(lay, i) : 0;
    const int stride = lay.mrope ? 3 : 1;
    cs[e] = rope_phase(a.freq.q[i], __ldg(a.positions + (t0 + t) * stride + axis));
  }
  if (tid < nt) {
    const int req = __ldg(a.req + t0 + tid), at = __ldg(a.tok + t0 + tid);
    const bool padding = req < 0;
    const bool bad = !padding && (req >= a.pool.num_reqs || at < 0 ||
                                  at >= (long long)a.pool.pt_stride * lay.page_size);
    if (bad) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
    live[tid] = !padding && !bad;
    slots[tid] = padding || bad ? -1 : slot_of(a.pool, lay.page_size, req, at, a.status);
  }
  __syncthreads();

  const long long layer_k = (long long)a.layer * a.pool.num_slots * lay.row_k;
  const long long slot = tk < nt ? slots[tk] : -1;
  const bool write_q = tk < nt && live[tk];
  const bool norms = gqa && (a.q_weight || a.k_weight);
  const float2 *c = cs + tk * np;
  float2 ph[8];  // NeoX pairs 8 q ..; interleaved pairs of chunk a, then of chunk b: the same ones
#pragma unroll
  for (int e = 0; e < 8; ++e) ph[e] = mine ? c[8 * q + e] : make_float2(1.f, 0.f);
  for (int base = 0; base < per_tok; base += groups * kBatch) {  // whole warps iterate alike
    if (base > 0) load(base + h_first);
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = base + h_first + j * groups;
      const bool isq = h < a.hq;
      float xa[8], xb[8];
      unpack8(ra[j], xa);
      unpack8(rb[j], xb);
      if (norms) {  // every lane takes part in the reduction
        const __nv_bfloat16 *wt = isq ? a.q_weight : a.k_weight;
        auto mean_sq = [&]() {
          float s = sum_sq8(xa) + sum_sq8(xb);
          for (int o = w >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
          return s / (float)band;
        };
        float mean = mean_sq() + a.eps;
        const float f = wt && h < per_tok ? norm_scale(mean) : 1.f;
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
      if (!mine || h >= per_tok || (isq ? !write_q : slot < 0)) continue;
      if (neox) {
#pragma unroll
        for (int e = 0; e < 8; ++e) rot_pair(xa[e], xb[e], ph[e]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; e += 2) {
          rot_pair(xa[e], xa[e + 1], ph[e >> 1]);
          rot_pair(xb[e], xb[e + 1], ph[4 + (e >> 1)]);
        }
      }
      __nv_bfloat16 *dst = (isq ? a.q_out + tok * a.q_out_stride
                                : a.pool.k + layer_k + slot * lay.row_k) +
                           column(h);
      st16(dst + ca, pack8_rn(xa));
      st16(dst + cb, pack8_rn(xb));
    }
  }

  if (gqa) {  // V rows, byte for byte: kThr / kTok threads to a token
    const int nc = lay.row_v >> 3, t = tid / (kThr / kTok);
    if (t >= nt || slots[t] < 0) return;
    const __nv_bfloat16 *src = a.v + (t0 + t) * a.v_stride;
    __nv_bfloat16 *dst =
        a.pool.v + ((long long)a.layer * a.pool.num_slots + slots[t]) * lay.row_v;
    for (int e = tid % (kThr / kTok); e < nc; e += kThr / kTok * kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (e + j * (kThr / kTok) < nc) v[j] = ld16(src + 8 * (e + j * (kThr / kTok)));
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (e + j * (kThr / kTok) < nc) st16(dst + 8 * (e + j * (kThr / kTok)), v[j]);
    }
    return;
  }
  // MLA: the latent rows, a warp to a token
  const int nc = lay.latent >> 3;
  for (int t = warp; t < nt; t += kThr / 32) {
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
    for (int c = lane; c < nc; c += 32) {  // read again, from L1
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
  // and the queries' latent parts, byte for byte: rows of nc chunks dealt to the warps
  if (a.q_out == a.q) return;
  const int rows = nt * a.hq;
  for (int i0 = warp; i0 < rows; i0 += kThr / 32 * kBatch) {
    for (int c = lane; c < nc; c += 64) {
      uint4 v[kBatch][2];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * (kThr / 32), t = i / a.hq;
        const __nv_bfloat16 *src = a.q + (t0 + t) * a.q_stride + (i - t * a.hq) * lay.row_k;
        if (i < rows && live[t]) {
          v[j][0] = ld16(src + 8 * c);
          if (c + 32 < nc) v[j][1] = ld16(src + 8 * (c + 32));
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * (kThr / 32), t = i / a.hq;
        __nv_bfloat16 *dst = a.q_out + (t0 + t) * a.q_out_stride + (i - t * a.hq) * lay.row_k;
        if (i < rows && live[t]) {
          st16(dst + 8 * c, v[j][0]);
          if (c + 32 < nc) st16(dst + 8 * (c + 32), v[j][1]);
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, cudaStream_t s) {
  // a token to a CTA while that gives every SM no more than a few CTAs, else four
  if (a.T <= 4 * kSms)
    append_kernel<1><<<(unsigned)a.T, kThr, 0, s>>>(a);
  else
    append_kernel<4><<<(unsigned)((a.T + 3) / 4), kThr, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kamera
