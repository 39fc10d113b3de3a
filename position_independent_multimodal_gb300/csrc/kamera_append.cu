// New tokens into the paged pool: the per-head RMS norm of queries and keys, their rotation to
// the tokens' positions and the write of K and V to the tokens' slots, in one pass.
//
//   GQA: q' = R(p) (q * rsqrt(mean q^2 + eps) * w_q) per query head, k' likewise with w_k into
//        the K row, v copied into the V row.
//   MLA: the latent c_KV normed with w_k and the k_pe band rotated into the row; the queries
//        (absorbed form) keep their latent part and turn their rope band.
//
// W = 2^ceil(log2(band / 16)) lanes take one (token, head) item: a lane holds the two 8-column
// chunks of a column unit, which are closed under pairing, so the norm is one shuffle reduction
// over the W lanes and the rotation needs no exchange; the weights are folded into the rotation.
// Sums of squares, the norm and the rotation are float32; phases by the exact Q0.64 range
// reduction of the other kernels; each output is rounded to bf16 once.
//
// append_kernel: a CTA of 256 threads per kTok tokens. A group of W lanes stays with one token and
// takes several of its heads at a time, so that their loads are in flight together, before the
// phases and slots are known. Few tokens (latency: 8 us at 8 tokens), or long rows (the rule and
// its measurements are at launch_append).
// append_stream_kernel: a warp to a token, in CTAs that stay, each lane's next chunks arriving by
// cp.async while it works, two heads at a time (one at a time: 4 us more). 16381 tokens of 28/4
// heads of 128: 62 us, 302 MB moved, 4.9 TB/s (append_kernel 82 us); few warps fit, and the chain
// of a head's norm and rotation takes its time in each.
// Bound: HBM (every byte is read and written once) at many tokens, latency at few.
#include <mutex>

#include "kamera_dev.cuh"
#include "kamera_ptx.cuh"
#include "kamera_smem.cuh"

namespace kamera {

namespace {

constexpr int kThr = 256;
constexpr int kBatch = 4;  // query heads a group of lanes (rows a warp) has in flight

// Every load is an ordinary one: q_out may be q, and the kernels live beside the one before them in
// the stream, which may write the page table or any input until ptx::wait_for_previous returns.
__device__ __forceinline__ uint4 ld16(const __nv_bfloat16 *p) {
  return *reinterpret_cast<const uint4 *>(p);
}

__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 neg2(f32x2 a) { return a ^ 0x8000000080000000ull; }

// The first and second members of a unit's eight pairs, two pairs to a register. NeoX-half: chunk
// a holds the first members, chunk b the second; interleaved: neighbours, pairs 0-3 in chunk a.
struct Unit {
  f32x2 a[4], b[4];
};

template <bool kNeox>
__device__ __forceinline__ Unit unpack_unit(const uint4 &ca, const uint4 &cb) {
  const uint32_t x[8] = {ca.x, ca.y, ca.z, ca.w, cb.x, cb.y, cb.z, cb.w};
  Unit u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kNeox) {
      u.a[i] = bf2_to_f2(x[i]);
      u.b[i] = bf2_to_f2(x[4 + i]);
    } else {
      u.a[i] = f2(__uint_as_float(x[2 * i] << 16), __uint_as_float(x[2 * i + 1] << 16));
      u.b[i] = f2(__uint_as_float(x[2 * i] & 0xFFFF0000u),
                  __uint_as_float(x[2 * i + 1] & 0xFFFF0000u));
    }
  }
  return u;
}

template <bool kNeox>
__device__ __forceinline__ void pack_unit(const Unit &u, uint4 *ca, uint4 *cb) {
  uint32_t x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kNeox) {
      x[i] = f2_to_bf2(u.a[i]);
      x[4 + i] = f2_to_bf2(u.b[i]);
    } else {
      float a0, a1, b0, b1;
      f2_split(u.a[i], a0, a1);
      f2_split(u.b[i], b0, b1);
      x[2 * i] = pack2_rn(a0, b0);
      x[2 * i + 1] = pack2_rn(a1, b1);
    }
  }
  *ca = make_uint4(x[0], x[1], x[2], x[3]);
  *cb = make_uint4(x[4], x[5], x[6], x[7]);
}

// Rotation with the weights folded in: a' = a (w_a cos) - b (w_b sin), b' = b (w_b cos) + a (w_a
// sin); the norm's factor multiplies the results.
struct Turn {
  f32x2 ac[4], bs[4], bc[4], as[4];  // bs negated
};

template <bool kNeox>
__device__ __forceinline__ Turn make_turn(const float2 *ph, const __nv_bfloat16 *w, int ca,
                                          int cb) {
  Unit u;
#pragma unroll
  for (int i = 0; i < 4; ++i) u.a[i] = u.b[i] = f2(1.f, 1.f);
  if (w)
    u = unpack_unit<kNeox>(ld16(w + ca), ld16(w + cb));
  Turn t;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 p0 = ph[2 * i], p1 = ph[2 * i + 1];
    const f32x2 c = f2(p0.x, p1.x), s = f2(p0.y, p1.y);
    t.ac[i] = mul2(u.a[i], c);
    t.as[i] = mul2(u.a[i], s);
    t.bc[i] = mul2(u.b[i], c);
    t.bs[i] = neg2(mul2(u.b[i], s));
  }
  return t;
}

__device__ __forceinline__ void turn_unit(const Turn &t, Unit &u) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const f32x2 a = u.a[i], b = u.b[i];
    u.a[i] = fma2(a, t.ac[i], mul2(b, t.bs[i]));
    u.b[i] = fma2(b, t.bc[i], mul2(a, t.as[i]));
  }
}

__device__ __forceinline__ void scale_unit(Unit &u, float f) {
  const f32x2 f2f = f2(f, f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    u.a[i] = mul2(u.a[i], f2f);
    u.b[i] = mul2(u.b[i], f2f);
  }
}

// Sum of squares of a unit, and over its group of w lanes.
__device__ __forceinline__ float sum_sq16(const Unit &u) {
  f32x2 s = f2(0.f, 0.f), v = s;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fma2(u.a[i], u.a[i], s);
    v = fma2(u.b[i], u.b[i], v);
  }
  float lo, hi;
  f2_split(add2(s, v), lo, hi);
  return lo + hi;
}
__device__ __forceinline__ float unit_sum_sq(const Unit &u, int w) {
  float s = sum_sq16(u);
  for (int o = w >> 1; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  return s;
}

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

__device__ __forceinline__ void st16(__nv_bfloat16 *p, const uint4 &v) {
  *reinterpret_cast<uint4 *>(p) = v;
}

// One head of a unit's lanes: the norm, the rotation, the store to chunks da and db. Whole warps
// come here alike: every lane takes part in the reduction.
template <bool kNeox>
__device__ __forceinline__ void finish_head(const uint4 &x, const uint4 &y, const Turn &turn,
                                            bool norm, float eps, int w, float inv_band, bool write,
                                            __nv_bfloat16 *da, __nv_bfloat16 *db) {
  Unit u = unpack_unit<kNeox>(x, y);
  float r = 1.f;
  if (norm) {
    float mean = fmaf(unit_sum_sq(u, w), inv_band, eps);
    const float f = norm_scale(mean);
    if (__any_sync(0xffffffffu, f != 1.f)) {
      scale_unit(u, f);
      mean = fmaf(unit_sum_sq(u, w), inv_band, eps * f * f);
    }
    r = rsqrtf(mean);
  }
  if (!write) return;
  turn_unit(turn, u);
  if (norm) scale_unit(u, r);
  uint4 za, zb;
  pack_unit<kNeox>(u, &za, &zb);
  st16(da, za);
  st16(db, zb);
}

// Two heads of a unit's lanes, the second one's chunks `step` columns behind the first's, with
// their reductions in flight together (chunks a and b of each in x).
template <bool kNeox>
__device__ __forceinline__ void finish_two(const uint4 (&x)[4], const Turn &turn, bool norm,
                                           float eps, int w, float inv_band, bool write0,
                                           bool write1, __nv_bfloat16 *da, __nv_bfloat16 *db,
                                           int step) {
  Unit u = unpack_unit<kNeox>(x[0], x[1]), v = unpack_unit<kNeox>(x[2], x[3]);
  float ru = 1.f, rv = 1.f;
  if (norm) {
    float su = sum_sq16(u), sv = sum_sq16(v);
    for (int o = w >> 1; o > 0; o >>= 1) {
      const float tu = __shfl_xor_sync(0xffffffffu, su, o);
      const float tv = __shfl_xor_sync(0xffffffffu, sv, o);
      su += tu;
      sv += tv;
    }
    su = fmaf(su, inv_band, eps);
    sv = fmaf(sv, inv_band, eps);
    const float fu = norm_scale(su), fv = norm_scale(sv);
    if (__any_sync(0xffffffffu, fu != 1.f || fv != 1.f)) {
      scale_unit(u, fu);
      scale_unit(v, fv);
      su = fmaf(unit_sum_sq(u, w), inv_band, eps * fu * fu);
      sv = fmaf(unit_sum_sq(v, w), inv_band, eps * fv * fv);
    }
    ru = rsqrtf(su);
    rv = rsqrtf(sv);
  }
  uint4 za, zb;
  if (write0) {
    turn_unit(turn, u);
    if (norm) scale_unit(u, ru);
    pack_unit<kNeox>(u, &za, &zb);
    st16(da, za);
    st16(db, zb);
  }
  if (write1) {
    turn_unit(turn, v);
    if (norm) scale_unit(v, rv);
    pack_unit<kNeox>(v, &za, &zb);
    st16(da + step, za);
    st16(db + step, zb);
  }
}

// Whether the queries' latent parts are to be copied; whether by every second CTA of append_kernel,
// beside the others' arithmetic. With the latter MLA with 16 heads takes 11 us instead of 13 at 150
// tokens, 13 instead of 15 at 600, 47 instead of 48 at 5003 and 113 instead of 109 at 12000.
__host__ __device__ inline bool copies_latents(const AppendArgs &a) {
  return a.lay.kind == KAMERA_MLA && a.hq > 0 && a.q_out != a.q;
}
__host__ __device__ inline bool copies_beside(const AppendArgs &a) {
  return copies_latents(a) && a.T <= 48 * kSms;
}

// The queries' latent parts of tokens t0 .. t0 + nt - 1, byte for byte: rows of nc chunks dealt to
// the CTA's warps.
__device__ __forceinline__ void copy_latents(const AppendArgs &a, long long t0, int nt,
                                             const int *live) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rows = nt * a.hq, nc = a.lay.latent >> 3;
  for (int i0 = warp; i0 < rows; i0 += kThr / 32 * kBatch) {
    for (int c = lane; c < nc; c += 64) {
      uint4 v[kBatch][2];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * (kThr / 32), t = i / a.hq;
        const __nv_bfloat16 *src = a.q + (t0 + t) * a.q_stride + (i - t * a.hq) * a.lay.row_k;
        if (i < rows && live[t]) {
          v[j][0] = ld16(src + 8 * c);
          if (c + 32 < nc) v[j][1] = ld16(src + 8 * (c + 32));
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int i = i0 + j * (kThr / 32), t = i / a.hq;
        __nv_bfloat16 *dst = a.q_out + (t0 + t) * a.q_out_stride + (i - t * a.hq) * a.lay.row_k;
        if (i < rows && live[t]) {
          st16(dst + 8 * c, v[j][0]);
          if (c + 32 < nc) st16(dst + 8 * (c + 32), v[j][1]);
        }
      }
    }
  }
}

template <int kTok, bool kNeox>
__global__ void __launch_bounds__(kThr, 2) append_kernel(const __grid_constant__ AppendArgs a) {
  __shared__ float2 cs[kTok * kMaxPairs];
  __shared__ long long slots[kTok];  // -1: no slot, K and V are not written
  __shared__ int live[kTok];         // 0: padding or a bad token, nothing is written
  ptx::launch_dependents();
  ptx::wait_for_previous();
  const DevLayout &lay = a.lay;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool copies = copies_beside(a);
  const long long t0 = (long long)(copies ? blockIdx.x >> 1 : blockIdx.x) * kTok;
  const int nt = (int)min((long long)kTok, a.T - t0);
  const int np = lay.npairs;
  const bool gqa = lay.kind == KAMERA_GQA;

  auto in_table = [&](int req, int at) {
    return req < a.pool.num_reqs && at >= 0 &&
           at < (long long)a.pool.pt_stride * lay.page_size;
  };
  if (copies && (blockIdx.x & 1)) {
    if (tid < nt) {
      const int req = a.req[t0 + tid];
      live[tid] = req >= 0 && in_table(req, a.tok[t0 + tid]);
    }
    __syncthreads();
    copy_latents(a, t0, nt, live);
    return;
  }

  // this group's token, its query heads and key bands h_first, h_first + groups, ...
  const int band = lay.rope_d, units = band >> 4;
  const int wsh = units <= 1 ? 0 : 32 - __clz(units - 1), w = 1 << wsh;
  const int q = tid & (w - 1), groups = kThr / kTok >> wsh;  // groups of lanes per token
  const int tk = tid / (kThr / kTok), h_first = (tid - tk * (kThr / kTok)) >> wsh;
  const int ca = kNeox ? 8 * q : 16 * q, cb = kNeox ? ca + (band >> 1) : ca + 8;
  const bool mine = q < units && tk < nt;
  const int n_k = gqa ? lay.H : 1;
  // the bands' columns: head h at off + h * pitch
  const int pitch = gqa ? lay.hd : lay.row_k, off = gqa ? 0 : lay.latent;
  const __nv_bfloat16 *qrow = a.q + (t0 + tk) * a.q_stride + off;
  const __nv_bfloat16 *krow = a.k + (t0 + tk) * a.k_stride + off;
  // the tokens' places first: their slots take two dependent loads
  int req = -1, at = 0;
  if (tid < nt) {
    req = a.req[t0 + tid];
    at = a.tok[t0 + tid];
  }
  uint4 ra[kBatch], rb[kBatch], ka, kb;
  auto load = [&](const __nv_bfloat16 *row, int h, int n, uint4 &x, uint4 &y) {
    x = y = make_uint4(0, 0, 0, 0);
    if (mine && h < n) {
      x = ld16(row + h * pitch + ca);
      y = ld16(row + h * pitch + cb);
    }
  };
#pragma unroll
  for (int j = 0; j < kBatch; ++j) load(qrow, h_first + j * groups, a.hq, ra[j], rb[j]);
  load(krow, h_first, n_k, ka, kb);
  // V: kThr / kTok threads to a token, the first chunk of each
  constexpr int kVThr = kThr / kTok;
  const int nv = gqa ? lay.row_v >> 3 : 0, ve = tid - tk * kVThr;
  uint4 v0;
  if (tk < nt && ve < nv) v0 = ld16(a.v + (t0 + tk) * a.v_stride + 8 * ve);
  if (tid < nt) {
    const bool padding = req < 0;
    const bool bad = !padding && !in_table(req, at);
    if (bad) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
    live[tid] = !padding && !bad;
    slots[tid] = padding || bad ? -1 : slot_of<false>(a.pool, lay.page_size, req, at, a.status);
  }

  for (int e = tid; e < nt * np; e += kThr) {
    const int t = e / np, i = e - t * np;
    const int axis = lay.mrope ? mrope_axis(lay, i) : 0;
    const int stride = lay.mrope ? 3 : 1;
    cs[e] = rope_phase(a.freq.q[i], a.positions[(t0 + t) * stride + axis]);
  }
  __syncthreads();

  const long long layer_k = (long long)a.layer * a.pool.num_slots * lay.row_k;
  const float2 *ph = cs + (mine ? tk * np + 8 * q : 0);
  auto finish = [&](const uint4 &x, const uint4 &y, const Turn &turn, bool norm, bool write,
                    __nv_bfloat16 *dst) {
    finish_head<kNeox>(x, y, turn, norm, a.eps, w, 1.f / (float)band, write, dst + ca, dst + cb);
  };
  if (a.hq > 0) {
    const Turn turn = make_turn<kNeox>(ph, a.q_weight, mine ? ca : 0, mine ? cb : 8);
    const bool write = mine && live[tk], norm = a.q_weight != nullptr;
    __nv_bfloat16 *dst = a.q_out + (t0 + tk) * a.q_out_stride + off;
    for (int base = h_first; base < a.hq + h_first; base += groups * kBatch) {
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int h = base + j * groups;
        if (base > h_first) load(qrow, h, a.hq, ra[j], rb[j]);
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int h = base + j * groups;
        finish(ra[j], rb[j], turn, norm, write && h < a.hq, dst + h * pitch);
      }
    }
  }
  {
    const bool norm = gqa && a.k_weight;
    const Turn turn =
        make_turn<kNeox>(ph, norm ? a.k_weight : nullptr, mine ? ca : 0, mine ? cb : 8);
    const bool write = mine && slots[tk] >= 0;
    __nv_bfloat16 *dst = a.pool.k + layer_k + (write ? slots[tk] * lay.row_k : 0) + off;
    for (int h = h_first; h < n_k + h_first; h += groups) {
      if (h > h_first) load(krow, h, n_k, ka, kb);
      finish(ka, kb, turn, norm, write && h < n_k, dst + h * pitch);
    }
  }

  if (gqa) {  // V rows, byte for byte
    if (tk >= nt || slots[tk] < 0) return;
    const __nv_bfloat16 *src = a.v + (t0 + tk) * a.v_stride;
    __nv_bfloat16 *dst =
        a.pool.v + ((long long)a.layer * a.pool.num_slots + slots[tk]) * lay.row_v;
    if (ve < nv) st16(dst + 8 * ve, v0);
    for (int e = ve + kVThr; e < nv; e += kVThr * kBatch) {
      uint4 v[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (e + j * kVThr < nv) v[j] = ld16(src + 8 * (e + j * kVThr));
#pragma unroll
      for (int j = 0; j < kBatch; ++j)
        if (e + j * kVThr < nv) st16(dst + 8 * (e + j * kVThr), v[j]);
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
        unpack8(ld16(a.k_weight + 8 * c), wv);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * f * r * wv[e];
        v = pack8_rn(x);
      }
      st16(dst + 8 * c, v);
    }
  }
  if (copies_latents(a) && !copies) copy_latents(a, t0, nt, live);
}

// ---------------------------------------------------------------------------------------
// Many tokens: a warp to a token, in CTAs that stay. A warp's lanes copy the 16-byte chunks that
// they will themselves use of its next token by cp.async while it works on this one, so nothing
// waits for another warp; the next token's page entry and position are on their way too. A lane
// has the same column unit in all its heads, so phases and weights are folded once a token.
// Bound: HBM.
// ---------------------------------------------------------------------------------------

constexpr int kStreamRoom = 214 * 1024;  // shared memory for the rows in flight (phases: 12 KB)
constexpr int kStreamWarps = 12;         // warps of a CTA at most (and 168 registers a thread)
constexpr int kStreamLeast = 6;          // and at least: fewer are slower than the CTA kernel

// Chunks of a token that a lane brings: two for each query head and key band of its group, then
// V chunks (GQA) or the latent rows' (MLA: of the token, of its query heads).
struct StreamPlan {
  int q, k, v, lk, lq;  // first chunk of each kind
  int chunks;           // in all
  int warps;            // of a CTA, as many as fit
};

StreamPlan stream_plan(const DevLayout &l, int hq, bool copy_q) {
  const int units = l.rope_d >> 4;
  int w = 1;
  while (w < units) w <<= 1;
  const int groups = 32 / w, n_k = l.kind == KAMERA_GQA ? l.H : 1;
  const int latent = ((l.latent >> 3) + 31) / 32;
  StreamPlan p;
  int n = 0;
  p.q = n;
  n += 2 * ((hq + groups - 1) / groups);
  p.k = n;
  n += 2 * ((n_k + groups - 1) / groups);
  p.v = n;
  if (l.kind == KAMERA_GQA) n += ((l.row_v >> 3) + 31) / 32;
  p.lk = n;
  n += latent;
  p.lq = n;
  if (l.kind == KAMERA_MLA && copy_q) n += latent * hq;
  p.chunks = n;
  p.warps = kStreamRoom / (2 * n * 512);
  if (p.warps > kStreamWarps) p.warps = kStreamWarps;
  return p;
}

template <bool kNeox>
__global__ void __launch_bounds__(32 * kStreamWarps, 1) append_stream_kernel(
    const __grid_constant__ AppendArgs a, const StreamPlan sp) {
  extern __shared__ __align__(16) unsigned char smem[];  // [warps][2][chunks][32] of 16 bytes
  __shared__ float2 phases[kStreamWarps][kMaxPairs];
  ptx::launch_dependents();
  ptx::wait_for_previous();
  const DevLayout &lay = a.lay;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int np = lay.npairs;
  const bool gqa = lay.kind == KAMERA_GQA;
  const int band = lay.rope_d, units = band >> 4;
  const int wsh = units <= 1 ? 0 : 32 - __clz(units - 1), w = 1 << wsh;
  const int q = lane & (w - 1), groups = 32 >> wsh, h_first = lane >> wsh;
  const bool unit = q < units;
  const int ca = unit ? (kNeox ? 8 * q : 16 * q) : 0;
  const int cb = unit ? (kNeox ? ca + (band >> 1) : ca + 8) : 8;
  const int n_k = gqa ? lay.H : 1, nv = gqa ? lay.row_v >> 3 : 0, nc = lay.latent >> 3;
  const int pitch = gqa ? lay.hd : lay.row_k, off = gqa ? 0 : lay.latent;
  const float inv_band = 1.f / (float)band;
  const long long layer_k = (long long)a.layer * a.pool.num_slots * lay.row_k;
  const long long layer_v = (long long)a.layer * a.pool.num_slots * lay.row_v;
  const bool copy_q = !gqa && a.q_out != a.q;
  const uint32_t stage = (uint32_t)sp.chunks * 512;
  unsigned char *const mem = smem + warp * 2 * stage + 16 * lane;
  const uint32_t sb = ptx::smem_addr(mem);
  float2 *const cs = phases[warp];
  auto copy = [&](uint32_t buf, int chunk, const __nv_bfloat16 *src) {
    ptx::cp_async16(sb + buf + chunk * 512, src, 16);
  };
  auto chunk = [&](uint32_t buf, int c) {
    return *reinterpret_cast<const uint4 *>(mem + buf + c * 512);
  };
  auto band_chunk = [&](uint32_t buf, int c) {  // zero where the lane has no unit: it is summed
    return unit ? chunk(buf, c) : make_uint4(0, 0, 0, 0);
  };
  // a token's rows into a buffer (its offset)
  auto fetch = [&](long long t, uint32_t buf) {
    if (t < a.T) {
      const __nv_bfloat16 *qr = a.q + t * a.q_stride, *kr = a.k + t * a.k_stride;
      if (unit) {
        const __nv_bfloat16 *p = qr + off + h_first * pitch;
        for (int h = h_first, c = sp.q; h < a.hq; h += groups, c += 2, p += groups * pitch) {
          copy(buf, c, p + ca);
          copy(buf, c + 1, p + cb);
        }
        p = kr + off + h_first * pitch;
        for (int h = h_first, c = sp.k; h < n_k; h += groups, c += 2, p += groups * pitch) {
          copy(buf, c, p + ca);
          copy(buf, c + 1, p + cb);
        }
      }
      const __nv_bfloat16 *vr = a.v + t * a.v_stride;
      for (int e = lane, c = sp.v; e < nv; e += 32, ++c) copy(buf, c, vr + 8 * e);
      if (!gqa) {
        for (int e = lane, c = sp.lk; e < nc; e += 32, ++c) copy(buf, c, kr + 8 * e);
        if (copy_q) {
          int c = sp.lq;
          for (int h = 0; h < a.hq; ++h)
            for (int e = lane; e < nc; e += 32, ++c) copy(buf, c, qr + h * lay.row_k + 8 * e);
        }
      }
    }
    ptx::cp_async_commit();
  };
  // what a token's place and phases are made of, fetched ahead; every lane has the same place
  struct Place {
    int req, tok;
  };
  auto load_place = [&](long long t) {
    Place p{-1, 0};
    if (t < a.T) {
      p.req = a.req[t];
      p.tok = a.tok[t];
    }
    return p;
  };
  auto load_page = [&](Place &p) {  // a place outside the table becomes padding, and is reported
    if (p.req < 0) return 0;
    if (p.req >= a.pool.num_reqs || p.tok < 0 ||
        p.tok >= (long long)a.pool.pt_stride * lay.page_size) {
      if (lane == 0) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
      p.req = -1;
      return 0;
    }
    return a.pool.pt[(long long)p.req * a.pool.pt_stride + p.tok / lay.page_size];
  };
  constexpr int kPos = kMaxPairs / 32;  // lane e makes pairs e, e + 32, ...
  long long pos[kPos];
  auto load_pos = [&](long long t) {
#pragma unroll
    for (int j = 0; j < kPos; ++j) {
      const int i = lane + 32 * j;
      if (i >= np || t >= a.T) continue;
      pos[j] = a.positions[lay.mrope ? 3 * t + mrope_axis(lay, i) : t];
    }
  };

  const long long step = (long long)gridDim.x * sp.warps;
  long long t = (long long)warp * gridDim.x + blockIdx.x;
  fetch(t, 0);
  Place now = load_place(t), next = load_place(t + step);
  load_pos(t);
  int page = load_page(now);
  for (uint32_t buf = 0; t < a.T; t += step, buf ^= stage) {
    fetch(t + step, buf ^ stage);
    // this token's slot and phases; the next one's page entry and position
    long long slot = -1;
    if (now.req >= 0) {
      if (page < 0 || ((long long)page + 1) * lay.page_size > a.pool.num_slots) {
        if (lane == 0) atomicOr(a.status, KAMERA_DEVICE_SLOT_OOB);
      } else {
        slot = (long long)page * lay.page_size + now.tok % lay.page_size;
      }
    }
    const bool live = now.req >= 0;
    __syncwarp();  // the last token's phases have been read
#pragma unroll
    for (int j = 0; j < kPos; ++j)
      if (lane + 32 * j < np) cs[lane + 32 * j] = rope_phase(a.freq.q[lane + 32 * j], pos[j]);
    page = load_page(next);
    now = next;
    next = load_place(t + 2 * step);
    load_pos(t + step);
    ptx::cp_async_wait_group1();  // this lane's chunks of the token
    __syncwarp();
    if (!live) continue;
    const float2 *ph = cs + (unit ? 8 * q : 0);
    if (a.hq > 0) {
      const Turn turn = make_turn<kNeox>(ph, a.q_weight, ca, cb);
      const bool norm = a.q_weight != nullptr;
      __nv_bfloat16 *dst = a.q_out + t * a.q_out_stride + off + h_first * pitch;
      // lanes of other groups may be out of heads a turn earlier: they take part all the same
      int h = h_first, c = sp.q;
      for (; h + groups < a.hq + h_first; h += 2 * groups, c += 4, dst += 2 * groups * pitch) {
        const uint4 x[4] = {band_chunk(buf, c), band_chunk(buf, c + 1), band_chunk(buf, c + 2),
                            band_chunk(buf, c + 3)};
        finish_two<kNeox>(x, turn, norm, a.eps, w, inv_band, unit && h < a.hq,
                          unit && h + groups < a.hq, dst + ca, dst + cb, groups * pitch);
      }
      if (h < a.hq + h_first)
        finish_head<kNeox>(band_chunk(buf, c), band_chunk(buf, c + 1), turn, norm, a.eps, w,
                           inv_band, unit && h < a.hq, dst + ca, dst + cb);
    }
    if (slot >= 0) {
      const bool norm = gqa && a.k_weight;
      const Turn turn = make_turn<kNeox>(ph, norm ? a.k_weight : nullptr, ca, cb);
      __nv_bfloat16 *row = a.pool.k + layer_k + slot * lay.row_k;
      __nv_bfloat16 *dst = row + off + h_first * pitch;
      for (int h = h_first, c = sp.k; h < n_k + h_first; h += groups, c += 2, dst += groups * pitch)
        finish_head<kNeox>(band_chunk(buf, c), band_chunk(buf, c + 1), turn, norm, a.eps, w,
                           inv_band, unit && h < n_k, dst + ca, dst + cb);
      for (int e = lane, c = sp.v; e < nv; e += 32, ++c)
        st16(a.pool.v + layer_v + slot * lay.row_v + 8 * e, chunk(buf, c));
      if (!gqa) {
        float r = 1.f, f = 1.f;
        if (a.k_weight) {
          auto mean_sq = [&]() {
            float s = 0.f;
            for (int e = lane, c = sp.lk; e < nc; e += 32, ++c) {
              float x[8];
              unpack8(chunk(buf, c), x);
#pragma unroll
              for (int i = 0; i < 8; ++i) x[i] *= f;
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
        for (int e = lane, c = sp.lk; e < nc; e += 32, ++c) {
          uint4 v = chunk(buf, c);
          if (a.k_weight) {
            float x[8], wv[8];
            unpack8(v, x);
            unpack8(ld16(a.k_weight + 8 * e), wv);
#pragma unroll
            for (int i = 0; i < 8; ++i) x[i] = x[i] * f * r * wv[i];
            v = pack8_rn(x);
          }
          st16(row + 8 * e, v);
        }
      }
    }
    if (copy_q) {
      __nv_bfloat16 *dst = a.q_out + t * a.q_out_stride;
      int c = sp.lq;
      for (int h = 0; h < a.hq; ++h, dst += lay.row_k)
        for (int e = lane; e < nc; e += 32, ++c) st16(dst + 8 * e, chunk(buf, c));
    }
  }
  ptx::cp_async_wait_all();
}

}  // namespace

namespace {

template <int kTok>
cudaError_t launch(const AppendArgs &a, cudaStream_t s) {
  const dim3 grid((unsigned)((a.T + kTok - 1) / kTok) * (copies_beside(a) ? 2 : 1));
  return launch_early(a.lay.style == KAMERA_ROPE_NEOX_HALF ? append_kernel<kTok, true>
                                                           : append_kernel<kTok, false>,
                      grid, kThr, 0, s, a);
}

}  // namespace

cudaError_t launch_append(const AppendArgs &a, cudaStream_t s) {
  // One token a CTA, four, or a warp a token, in us: calls one after another over 400 MB, from a
  // graph (in brackets how many warps fit):
  //                       T = 304          608          1216        2432        16381
  //                     one four warps  four warps   four warps  four warps  four warps
  //   28/4 x 128 (11)   6.3  6.1  6.9    6.8  7.4     8.6  9.0   15.9 15.0     85   62
  //   32/8 x 128 (8)    6.6  7.2  7.5    8.0  8.2    10.2 10.6   19.0 17.4    103   91
  //   40/8 x 128 (7)    6.7  8.6  8.0    9.6  8.9    11.9 15.6   22.1 22.9    122  106
  //   48/8 x 128 (6)                                 12.4 16.4   22.9 24.8    126  129
  //   56/8 x 128 (5)                                 13.5 17.3   24.1 32.6    131  164
  //   32/32 x 128 (4)   8.0 10.8 10.3   12.2 12.1    16.2 20.3   29.2 36.7    171  206
  //   6/2 x 64 (12)     5.5  4.9  4.6    5.0  4.6     5.6  4.9   10.4  7.1     68   33
  //   16/2 x 128 (12)   6.1  5.7  6.0    6.0  6.2     7.3  7.2   13.6 11.2     81   49
  //   MLA, in place (12) 6.4 6.0  5.3    6.4  5.6     7.5  6.6   13.2  9.2     81   40
  //   MLA, 10 copied (7)                             13.3 13.8   23.4 20.0    121   90
  //   MLA, 12 copied (6)                             13.6 14.5   24.1 21.0    127  108
  //   MLA, 16 copied (5) 11.3 6.5 8.8    7.6  9.6    14.1 16.1   25.5 29.9    140  149
  // CTAs of four tokens, two to an SM, are one wave up to 8 * kSms tokens (half as many with copies
  // beside them, which double the CTAs), and hard to beat until then; rows so narrow that all the
  // warps fit have more of them in flight as warps from the start. Six warps are the border: 15 %
  // faster for MLA, 2 to 8 % slower for GQA; fewer do not hold the rows in flight that HBM wants.
  const long long n = a.T * (copies_beside(a) ? 2 : 1);
  if (n <= 2 * kSms) return launch<1>(a, s);
  const StreamPlan sp = stream_plan(a.lay, a.hq, a.q_out != a.q);
  if (sp.warps < kStreamLeast || (sp.warps < kStreamWarps && n <= 8 * kSms)) return launch<4>(a, s);
  static int configured[64] = {0};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      e = cudaFuncSetAttribute(append_stream_kernel<true>,
                               cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamRoom);
      if (e == cudaSuccess)
        e = cudaFuncSetAttribute(append_stream_kernel<false>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamRoom);
      if (e != cudaSuccess) return e;
      configured[dev] = 1;
    }
  }
  const size_t bytes = (size_t)2 * sp.chunks * 512 * sp.warps;
  return launch_early(a.lay.style == KAMERA_ROPE_NEOX_HALF ? append_stream_kernel<true>
                                                           : append_stream_kernel<false>,
                      dim3(kSms), 32 * sp.warps, bytes, s, a, sp);
}

}  // namespace kamera
