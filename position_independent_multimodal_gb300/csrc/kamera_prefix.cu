// Decode attention of a batch whose requests share prefixes: each group's prefix is read once
// for all the group's query rows, the tokens after it for each request alone.
//   s_t = scale * q . K_t,  o = sum_t softmax(s)_t V_t,  lse = log sum_t exp(s_t)
// over tokens [0, ctx) of each request; the softmax over a union of token sets is the parts'
// softmaxes weighted by their masses, o = sum_i e^(lse_i - lse) o_i, lse = log sum_i e^(lse_i).
//
// prefix_plan_kernel lists the groups and requests with tokens and numbers their units
// (kamera_prefix.cuh), an attention kernel works the units off, prefix_merge_kernel joins the
// parts. This file has the attention kernel for any layout (CUDA cores); the layouts with
// tensor-core tiles take the kernel of kamera_prefix_tc.cu.
#include <mutex>

#include "kamera_prefix.cuh"
#include "kamera_smem.cuh"

namespace kamera {

namespace {

constexpr int kPlanThr = 1024;

// Inclusive scan over the CTA's threads; every thread also gets the total.
__device__ __forceinline__ long long plan_scan(long long x, long long *total) {
  __shared__ long long part[kPlanThr / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) part[warp] = x;
  __syncthreads();
  long long before = 0, sum = 0;
  for (int w = 0; w < kPlanThr / 32; ++w) {
    if (w < warp) before += part[w];
    sum += part[w];
  }
  *total = sum;
  return x + before;
}

__global__ void __launch_bounds__(kPlanThr) prefix_plan_kernel(const __grid_constant__ PrefixArgs a) {
  const PrefixPlan p = prefix_plan(a.ws, a.n_reqs, a.hq, a.dv, a.vh, a.rb, a.n_ctas);
  __shared__ int broken;
  const int tid = threadIdx.x, R = a.n_reqs, G = a.n_groups;
  const int hpk = a.hq / a.n_kv, blocks = a.n_kv * a.vh;
  const long long cap = (long long)a.pool.pt_stride * a.lay.page_size;
  if (tid == 0) broken = 0;
  __syncthreads();
  for (int g = tid; g <= G; g += kPlanThr) {
    const int s = a.group_start[g];
    if (s < 0 || s > R || (g == 0 && s != 0) || (g == G && s != R) ||
        (g > 0 && a.group_start[g - 1] > s))
      broken = 1;
  }
  __syncthreads();
  if (broken) {  // the groups do not partition the requests: nothing is written
    for (int r = tid; r < R; r += kPlanThr) p.req_state[r] = 0;
    if (tid < 8) p.head[tid] = 0;
    if (tid == 0) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
    return;
  }
  // requests: their group, whether they keep its rules, their tiles
  for (int g = tid; g < G; g += kPlanThr) p.lead[g] = 0x7FFFFFFF;
  __syncthreads();
  for (int r = tid; r < R; r += kPlanThr) {
    int lo = 0, hi = G - 1;  // the last group that starts at or before r (empty ones come first)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (a.group_start[mid] <= r)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int s0 = a.group_start[lo], prefix = a.prefix_len[lo], ctx = a.ctx_len[r];
    const bool wrong =
        prefix < 0 || prefix > cap || ctx < 0 || ctx > cap || (ctx > 0 && ctx < prefix);
    if (wrong) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
    const bool active = !wrong && ctx > 0;
    if (active) atomicMin(p.lead + lo, r);
    p.req_state[r] = !wrong;
    p.req_group[r] = active ? lo : -1;
    p.req_at[r] = r - s0;
    p.req_size[r] = a.group_start[lo + 1] - s0;
    p.req_tiles[r] = active ? ceil_div(prefix, a.tile) : 0;
    p.req_own[r] = active ? tiles_of(prefix, ctx, a.tile) : 0;
  }
  __syncthreads();
  // groups: units of each prefix
  long long base = 0, listed = 0;
  for (int g0 = 0; g0 < G; g0 += kPlanThr) {
    const int g = g0 + tid;
    int s0 = 0, n = 0, prefix = 0, lead = 0x7FFFFFFF;
    long long units = 0;
    if (g < G) {
      s0 = a.group_start[g];
      n = a.group_start[g + 1] - s0;
      prefix = a.prefix_len[g];
      lead = __ldcg(p.lead + g);
      if (lead != 0x7FFFFFFF && prefix > 0)
        units = (long long)blocks * ceil_div(n * hpk, a.rb) * ceil_div(prefix, a.tile);
    }
    long long total, count;
    const long long at = base + plan_scan(units, &total) - units;
    const long long k = listed + plan_scan(units > 0, &count) - (units > 0);
    if (g < G) {
      p.gr_u0[g] = units > 0 ? at : -1;
      if (units > 0) {
        p.g_u0[k] = at;
        p.g_list[k] = s0;
        p.g_size[k] = n;
        p.g_prefix[k] = prefix;
        p.g_lead[k] = lead;
      }
    }
    base += total;
    listed += count;
  }
  __syncthreads();
  const long long prefix_units = base, groups = listed;
  // requests: units of their own tokens
  listed = 0;
  for (int r0 = 0; r0 < R; r0 += kPlanThr) {
    const int r = r0 + tid;
    const int tiles = r < R ? p.req_own[r] : 0, g = r < R ? p.req_group[r] : -1;
    const long long units = (long long)blocks * ceil_div(hpk, a.rb) * tiles;
    long long total, count;
    const long long at = base + plan_scan(units, &total) - units;
    const long long k = listed + plan_scan(units > 0, &count) - (units > 0);
    if (r < R) {
      p.req_pu0[r] = g >= 0 ? p.gr_u0[g] : -1;
      p.req_ou0[r] = units > 0 ? at : -1;
      if (units > 0) {
        p.r_u0[k] = at;
        p.r_list[k] = r;
        p.r_from[k] = a.prefix_len[g];
        p.r_to[k] = a.ctx_len[r];
      }
    }
    base += total;
    listed += count;
  }
  if (tid == 0) {
    p.head[0] = base;
    p.head[1] = groups;
    p.head[2] = listed;
    p.head[3] = base < a.n_ctas ? base : a.n_ctas;
    p.head[4] = prefix_units;
  }
}

// ---------------------------------------------------------------------------------------
// Any layout, CUDA cores. A CTA of 256 threads works its segments off, up to 8 query rows a
// block and 256 tokens a tile. Scores: thread t owns token t of the tile, streams its K row
// (16-byte loads, eight in flight) against the rows' queries in shared memory. P·V: each thread
// owns an 8-column chunk of V and a subset of the tokens; the running sums stay in registers,
// rescaled when the running maximum rises, and are added up through shared memory at the end of
// a segment. Bound: FMA issue (8 rows reuse each K and V element), then HBM.
// ---------------------------------------------------------------------------------------

constexpr int kThr = 256;
constexpr int kTile = 256;
constexpr int kRows = 8;
constexpr int kBatch = 8;

struct GenPlan {
  int q;     // f32x2 [kRows][dk / 2]
  int p;     // float [kTile][kRows]
  int slot;  // long long [kTile]
  int red;   // float [lanes][kRows][dv]
  int stat;  // float m[kRows], l[kRows], f[kRows], warp partials [kRows][kThr / 32]
  int total;
};

__host__ __device__ inline GenPlan gen_plan(int dk, int dv) {
  GenPlan p;
  const int lanes = kThr / (dv / 8) > 0 ? kThr / (dv / 8) : 1;
  int o = 0;
  p.q = o;
  o += kRows * dk * 4;
  p.p = o;
  o += kRows * kTile * 4;
  p.slot = o;
  o += kTile * 8;
  p.red = o;
  o += lanes * kRows * dv * 4;
  p.stat = o;
  o += (3 * kRows + kRows * (kThr / 32)) * 4;
  p.total = o;
  return p;
}

__global__ void __launch_bounds__(kThr) prefix_gen_kernel(const __grid_constant__ PrefixArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  const GenPlan P = gen_plan(a.dk, a.dv);
  const PrefixPlan plan = prefix_plan(a.ws, a.n_reqs, a.hq, a.dv, a.vh, a.rb, a.n_ctas);
  f32x2 *qs = reinterpret_cast<f32x2 *>(smem + P.q);
  float *ps = reinterpret_cast<float *>(smem + P.p);
  long long *slots = reinterpret_cast<long long *>(smem + P.slot);
  float *red = reinterpret_cast<float *>(smem + P.red);
  float *m = reinterpret_cast<float *>(smem + P.stat), *l = m + kRows, *f = l + kRows;
  float *wp = f + kRows;
  const DevLayout &lay = a.lay;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int dk = a.dk, dv = a.dv, dk2 = dk >> 1;
  const float neg_inf = -__int_as_float(0x7f800000);
  const int chunks = dv >> 3, lanes = kThr / chunks;
  const int c = tid % chunks, tl = tid / chunks;
  const bool gqa = lay.kind == KAMERA_GQA;
  SegmentWalk walk;
  walk.start(a, plan, blockIdx.x);
  Segment s;
  while (walk.next(a, plan, &s)) {
    __syncthreads();  // the last segment's shared memory has been read
    for (int e = tid; e < kRows * dk2; e += kThr) {
      const int g = e / dk2, d = 2 * (e - g * dk2);
      f32x2 v = f2(0.f, 0.f);
      if (g < s.rows) {
        int r, h;
        segment_row(a, s, g, &r, &h);
        const __nv_bfloat16 *q = a.q + ((long long)r * a.hq + h) * dk + d;
        v = f2(__bfloat162float(q[0]), __bfloat162float(q[1]));
      }
      qs[e] = v;
    }
    if (tid < kRows) {
      m[tid] = neg_inf;
      l[tid] = 0.f;
    }
    f32x2 o8[kRows][4];
#pragma unroll
    for (int g = 0; g < kRows; ++g)
#pragma unroll
      for (int e = 0; e < 4; ++e) o8[g][e] = f2(0.f, 0.f);
    const __nv_bfloat16 *kbase = a.pool.k + (long long)a.layer * a.pool.num_slots * lay.row_k +
                                 (gqa ? s.kvh * lay.hd : 0);
    const __nv_bfloat16 *vbase =
        gqa ? a.pool.v + (long long)a.layer * a.pool.num_slots * lay.row_v + s.kvh * lay.hd
            : a.pool.k + (long long)a.layer * a.pool.num_slots * lay.row_k;
    const int vrow = gqa ? lay.row_v : lay.row_k;
    for (int t0 = s.tok0, n; t0 < s.tok1; t0 += n) {
      n = min(kTile - t0 % kTile, s.tok1 - t0);
      __syncthreads();  // the last tile's slots and weights have been read
      const long long slot =
          tid < n ? slot_of(a.pool, lay.page_size, s.lead, (long long)t0 + tid, a.status) : -1;
      slots[tid] = slot;
      f32x2 acc[kRows];
#pragma unroll
      for (int g = 0; g < kRows; ++g) acc[g] = f2(0.f, 0.f);
      if (slot >= 0) {
        const __nv_bfloat16 *krow = kbase + slot * lay.row_k;
        for (int d0 = 0; d0 < dk; d0 += 8 * kBatch) {
          uint4 buf[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j)
            if (d0 + 8 * j < dk) buf[j] = __ldg(reinterpret_cast<const uint4 *>(krow + d0 + 8 * j));
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            if (d0 + 8 * j >= dk) break;
            const f32x2 x0 = bf2_to_f2(buf[j].x), x1 = bf2_to_f2(buf[j].y);
            const f32x2 x2 = bf2_to_f2(buf[j].z), x3 = bf2_to_f2(buf[j].w);
            const int pair = (d0 + 8 * j) >> 1;
#pragma unroll
            for (int g = 0; g < kRows; ++g) {
              const ulonglong2 qa = *reinterpret_cast<const ulonglong2 *>(qs + g * dk2 + pair);
              const ulonglong2 qb = *reinterpret_cast<const ulonglong2 *>(qs + g * dk2 + pair + 2);
              acc[g] = fma2(qa.x, x0, acc[g]);
              acc[g] = fma2(qa.y, x1, acc[g]);
              acc[g] = fma2(qb.x, x2, acc[g]);
              acc[g] = fma2(qb.y, x3, acc[g]);
            }
          }
        }
      }
      float sc[kRows];
#pragma unroll
      for (int g = 0; g < kRows; ++g) {
        float lo, hi;
        f2_split(acc[g], lo, hi);
        sc[g] = slot >= 0 ? (lo + hi) * a.scale : neg_inf;
        float w = sc[g];
        for (int o = 16; o > 0; o >>= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, o));
        if (lane == 0) wp[g * (kThr / 32) + warp] = w;
      }
      __syncthreads();
      if (tid < kRows) {
        float w = m[tid];
        for (int i = 0; i < kThr / 32; ++i) w = fmaxf(w, wp[tid * (kThr / 32) + i]);
        f[tid] = m[tid] > neg_inf ? expf(m[tid] - w) : 0.f;
        m[tid] = w;
      }
      __syncthreads();
#pragma unroll
      for (int g = 0; g < kRows; ++g) {
        // a score of NaN stays one; a row without a finite maximum has weights of zero
        const float e = slot >= 0 && !(m[g] == neg_inf && sc[g] == neg_inf) ? expf(sc[g] - m[g])
                                                                            : 0.f;
        ps[tid * kRows + g] = e;
        float w = e;
        for (int o = 16; o > 0; o >>= 1) w += __shfl_xor_sync(0xffffffffu, w, o);
        if (lane == 0) wp[g * (kThr / 32) + warp] = w;
      }
      __syncthreads();
      if (tid < kRows) {
        float w = 0.f;
        for (int i = 0; i < kThr / 32; ++i) w += wp[tid * (kThr / 32) + i];
        l[tid] = l[tid] * f[tid] + w;
      }
      if (tl < lanes) {
#pragma unroll
        for (int g = 0; g < kRows; ++g) {
          const f32x2 ff = f2(f[g], f[g]);
#pragma unroll
          for (int e = 0; e < 4; ++e) o8[g][e] = fma2(ff, o8[g][e], f2(0.f, 0.f));
        }
        for (int t = tl; t < n; t += lanes * kBatch) {
          uint4 buf[kBatch];
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int tt = t + j * lanes;
            const long long st = tt < n ? slots[tt] : -1;
            if (st >= 0) buf[j] = __ldg(reinterpret_cast<const uint4 *>(vbase + st * vrow + 8 * c));
          }
#pragma unroll
          for (int j = 0; j < kBatch; ++j) {
            const int tt = t + j * lanes;
            if (tt >= n || slots[tt] < 0) continue;
            const f32x2 x0 = bf2_to_f2(buf[j].x), x1 = bf2_to_f2(buf[j].y);
            const f32x2 x2 = bf2_to_f2(buf[j].z), x3 = bf2_to_f2(buf[j].w);
#pragma unroll
            for (int g = 0; g < kRows; ++g) {
              const float pg = ps[tt * kRows + g];
              const f32x2 pp = f2(pg, pg);
              o8[g][0] = fma2(pp, x0, o8[g][0]);
              o8[g][1] = fma2(pp, x1, o8[g][1]);
              o8[g][2] = fma2(pp, x2, o8[g][2]);
              o8[g][3] = fma2(pp, x3, o8[g][3]);
            }
          }
        }
      }
    }
    __syncthreads();
    if (tl < lanes) {
#pragma unroll
      for (int g = 0; g < kRows; ++g) {
        float4 *dst = reinterpret_cast<float4 *>(red + (tl * kRows + g) * dv + 8 * c);
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) f2_split(o8[g][e], v[2 * e], v[2 * e + 1]);
        dst[0] = make_float4(v[0], v[1], v[2], v[3]);
        dst[1] = make_float4(v[4], v[5], v[6], v[7]);
      }
    }
    __syncthreads();
    for (int e = tid; e < s.rows * dv; e += kThr) {
      const int g = e / dv, d = e - g * dv;
      float sum = 0.f;
      for (int i = 0; i < lanes; ++i) sum += red[(i * kRows + g) * dv + d];
      float *o, *lse;
      segment_out(a, plan, s, blockIdx.x, g, &o, &lse);
      o[d] = l[g] == 0.f ? 0.f : sum / l[g];
      if (d == 0) *lse = l[g] == 0.f ? neg_inf : m[g] + logf(l[g]);
    }
  }
}

// One warp per (request, query head, column half): the row's parts weighted by
// exp(lse_i - lse), rounded to bf16 once.
__global__ void __launch_bounds__(kThr) prefix_merge_kernel(const __grid_constant__ PrefixArgs a) {
  const PrefixPlan p = prefix_plan(a.ws, a.n_reqs, a.hq, a.dv, a.vh, a.rb, a.n_ctas);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long w = (long long)blockIdx.x * (kThr / 32) + warp;
  const long long n_rh = (long long)a.n_reqs * a.hq;
  if (w >= n_rh * a.vh) return;
  const long long rh = w / a.vh;
  const int half = (int)(w - rh * a.vh);
  const int r = (int)(rh / a.hq), h = (int)(rh - (long long)r * a.hq);
  if (!p.req_state[r]) return;
  const int hpk = a.hq / a.n_kv, kvh = h / hpk, dvh = a.dv / a.vh;
  const float neg_inf = -__int_as_float(0x7f800000);
  const long long U = p.head[0], n = p.head[3];
  // the two blocks of the row: first unit, tiles, index of the row in its block, carries
  int c0[2] = {0, 0}, nc[2] = {0, 0}, at[2] = {0, 0};
  bool have[2];
  float top = neg_inf;
  for (int b = 0; b < 2; ++b) {
    const long long base = b ? p.req_ou0[r] : p.req_pu0[r];
    have[b] = base >= 0;
    if (!have[b]) continue;
    const int tiles = b ? p.req_own[r] : p.req_tiles[r];
    const int row = (b ? 0 : p.req_at[r] * hpk) + (h - kvh * hpk);
    const int rows_all = (b ? 1 : p.req_size[r]) * hpk;
    const int nrb = ceil_div(rows_all, a.rb), blk = row / a.rb;
    at[b] = row - blk * a.rb;
    const long long u0 = base + (((long long)kvh * a.vh + half) * nrb + blk) * tiles;
    const long long u1 = u0 + tiles;
    // CTAs that start inside the block: c U / n in (u0, u1)
    long long lo = u0 * n / U;
    while (lo * U / n <= u0) ++lo;
    long long hi = lo;
    while (hi < n && hi * U / n < u1) ++hi;
    c0[b] = (int)lo;
    nc[b] = (int)(hi - lo);
    top = fmaxf(top, p.home_lse[((long long)b * a.vh + half) * n_rh + rh]);
    for (int i = 0; i < nc[b]; ++i)
      top = fmaxf(top, p.carry_lse[(long long)(c0[b] + i) * a.rb + at[b]]);
  }
  float sum = 0.f;
  float acc[32];  // columns lane, lane + 32, ...
#pragma unroll
  for (int e = 0; e < 32; ++e) acc[e] = 0.f;
  for (int b = 0; b < 2; ++b) {
    if (!have[b]) continue;
    for (int i = -1; i < nc[b]; ++i) {
      const long long k = (long long)(c0[b] + i) * a.rb + at[b];
      const float z = i < 0 ? p.home_lse[((long long)b * a.vh + half) * n_rh + rh] : p.carry_lse[k];
      if (z == neg_inf) continue;  // nothing to add; a NaN goes on
      const float wt = expf(z - top);
      const float *o = i < 0 ? p.home_o + (b * n_rh + rh) * a.dv + half * dvh : p.carry_o + k * dvh;
      sum += wt;
#pragma unroll
      for (int e = 0; e < 32; ++e)
        if (lane + 32 * e < dvh) acc[e] = fmaf(wt, o[lane + 32 * e], acc[e]);
    }
  }
  const bool empty = sum == 0.f;
#pragma unroll
  for (int e = 0; e < 32; ++e)
    if (lane + 32 * e < dvh)
      a.out[rh * a.dv + half * dvh + lane + 32 * e] =
          __float2bfloat16_rn(empty ? 0.f : acc[e] / sum);
  if (lane == 0 && half == 0) a.lse[rh] = empty ? neg_inf : top + logf(sum);
}

}  // namespace

void prefix_shape(const DevLayout &l, int hq, int *rb, int *tile, int *vh, int *n_ctas) {
  if (prefix_tc_layout(l)) return prefix_tc_shape(l, hq, rb, tile, vh, n_ctas);
  *rb = kRows;
  *tile = kTile;
  *vh = 1;
  *n_ctas = 2 * kPrefixCtas;
}

size_t prefix_workspace(const DevLayout &l, long long n_reqs, int hq, int dv) {
  int rb, tile, vh, n;
  prefix_shape(l, hq, &rb, &tile, &vh, &n);
  return prefix_plan(nullptr, n_reqs, hq, dv, vh, rb, n).total;
}

cudaError_t launch_prefix_attention(const PrefixArgs &a, cudaStream_t s) {
  static int configured[64] = {0};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      e = cudaFuncSetAttribute(prefix_gen_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               gen_plan(1024, 1024).total);
      if (e == cudaSuccess) e = prepare_prefix_tc();
      if (e != cudaSuccess) return e;
      configured[dev] = 1;
    }
  }
  prefix_plan_kernel<<<1, kPlanThr, 0, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (prefix_tc_layout(a.lay)) {
    e = launch_prefix_tc(a, s);
  } else {
    prefix_gen_kernel<<<a.n_ctas, kThr, gen_plan(a.dk, a.dv).total, s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  const long long warps = (long long)a.n_reqs * a.hq * a.vh;
  prefix_merge_kernel<<<(unsigned)((warps + kThr / 32 - 1) / (kThr / 32)), kThr, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace kamera
