// Decode attention of a batch whose requests share prefixes: each group's prefix is read once
// for all the group's query rows, the tokens after it for each request alone.
//   s_t = scale * q . K_t,  o = sum_t softmax(s)_t V_t,  lse = log sum_t exp(s_t)
// over tokens [0, ctx) of each request; the softmax over a union of token sets is the parts'
// softmaxes weighted by their masses, o = sum_i e^(lse_i - lse) o_i, lse = log sum_i e^(lse_i).
//
// The kernels of a call start early, each while the one before it still runs, and wait for what
// they read: the attention kernels for the plan, the merge for the attention kernels. Where both
// of these run, the thin one works beside the wide one's last CTAs (it needs the plan alone, which
// is complete when every CTA of the wide one has let it start) and waits for it at its end.
//
// prefix_plan_kernel lists the groups and requests with tokens and numbers their units
// (kamera_prefix.cuh), the attention kernels work the units off, prefix_merge_kernel joins the
// parts. This file has the attention kernel for any layout (CUDA cores); GQA with head_dim 64 or
// 128 and MLA with 512 + 64 take those of kamera_prefix_tc.cu (wide blocks) and
// kamera_prefix_thin.cu.
#include <mutex>

#include "kamera_prefix.cuh"
#include "kamera_ptx.cuh"
#include "kamera_smem.cuh"

namespace kamera {

namespace {

constexpr int kPlanThr = 256;
// Tiles that a worker may have more than its equal part for each wide block to have workers of its
// own: blocks of two tiles of query rows, of one. Calls with workers of each block's own | with the
// units in equal parts, in us, by the tiles more:
//   two tiles of rows (28/4 heads of 128, 252 rows a block)
//     1: 59 | 66, 62 | 71   2: 83 | 91, 60 | 61   4: 82 | 85, 132 | 138   6: 90 | 93, 87 | 88
//     7: 136 | 138, 106 | 107, 110 | 106   8: 93 | 87   12: 138 | 136   16: 119 | 105
//   one tile (63 rows a block; MLA)
//     1: 39 | 45, 38 | 43, 77 | 71   2: 41 | 42, 48 | 48; 62 | 63, 95 | 99, 79 | 76
//     3: 55 | 55; 89 | 87, 97 | 91   4: 67 | 63, 73 | 71; 112 | 106   6: 74 | 69; 132 | 124
//     8: 67 | 60
constexpr int kOwnExtraTwo = 6, kOwnExtraOne = 2;
constexpr int kOwnRows = 128;    // query rows of a tile
constexpr int kPlanNear = 1024;  // groups and listed entries kept in shared memory

// Inclusive scans of N values at a time over the CTA's threads, in place; total: their sums.
template <int N>
__device__ __forceinline__ void plan_scan(long long (&x)[N], long long (&total)[N]) {
  __shared__ long long part[N][kPlanThr / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long y = __shfl_up_sync(0xffffffffu, x[k], o);
      if (lane >= o) x[k] += y;
    }
  __syncthreads();  // earlier readers of part are done
  if (lane == 31)
#pragma unroll
    for (int k = 0; k < N; ++k) part[k][warp] = x[k];
  __syncthreads();
  if (warp < N) {  // warp k scans the warps' sums of value k
    long long y = lane < kPlanThr / 32 ? part[warp][lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long z = __shfl_up_sync(0xffffffffu, y, o);
      if (lane >= o) y += z;
    }
    if (lane < kPlanThr / 32) part[warp][lane] = y;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    if (warp > 0) x[k] += part[k][warp - 1];
    total[k] = part[k][kPlanThr / 32 - 1];
  }
}

// Picks of the classes without an index into registers, which would put them into local memory.
template <class T>
__device__ __forceinline__ T by_class(int c, const T &wide, const T &thin) {
  return c ? thin : wide;
}
__device__ __forceinline__ PrefixPlan::Lists lists_of(const PrefixPlan &p, int c) {
  const PrefixPlan::Lists &a = p.cls[0], &b = p.cls[1];
  return {c ? b.g_u0 : a.g_u0,         c ? b.g_first : a.g_first,   c ? b.g_size : a.g_size,
          c ? b.g_prefix : a.g_prefix, c ? b.g_lead : a.g_lead,     c ? b.start : a.start,
          c ? b.carry_lse : a.carry_lse, c ? b.carry_o : a.carry_o};
}

// One CTA: checks the arguments, lists the groups and requests that have units, and finds each
// wide worker's first block. Bound: the latency of its few dependent steps (6 to 8 us for 4 to 128
// requests; 512 or 1024 threads are slower, by their barriers), and from some thousand requests its
// rounds of 256: 11 us for 1024 requests of one group, 104 for 16384; with a group to each request
// 15 and 265 us.
__global__ void __launch_bounds__(kPlanThr)
    prefix_plan_kernel(const __grid_constant__ PrefixArgs a) {
  ptx::launch_dependents();
  const PrefixPlan p = prefix_plan(a.shape, a.ws, a.n_reqs, a.hq, a.dv);
  __shared__ int near_start[kPlanNear + 1], near_lead[kPlanNear];
  __shared__ long long near_u0[kPlanNear], near_r[kPlanNear];  // of the wide class
  __shared__ int broken, worst, near_w0[kPlanThr], near_k[kPlanThr];
  const int tid = threadIdx.x, R = a.n_reqs, G = a.n_groups;
  const int hpk = a.hpk, own_cls = class_of(a.shape, hpk);
  const long long cap = (long long)a.pool.pt_stride * a.lay.page_size;
  const bool near_g = G <= kPlanNear;
  const int *start = near_g ? near_start : a.group_start;
  int *lead = near_g ? near_lead : p.lead;
  if (tid == 0) {
    broken = worst = 0;
    *p.gave_up = 0;
  }
  __syncthreads();
  for (int g = tid; g <= G; g += kPlanThr) {
    const int s = a.group_start[g];
    if (near_g) near_start[g] = s;
    if (g < G) lead[g] = 0x7FFFFFFF;
    if (s < 0 || s > R || (g == 0 && s != 0) || (g == G && s != R) ||
        (g > 0 && a.group_start[g - 1] > s))
      broken = 1;
  }
  __syncthreads();
  if (broken) {  // the groups do not partition the requests: nothing is written
    for (int r = tid; r < R; r += kPlanThr) p.req_state[r] = 0;
    if (tid <= 16) p.head[tid] = 0;
    if (tid == 0) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
    return;
  }
  // requests: their group, whether they keep its rules
  for (int r = tid; r < R; r += kPlanThr) {
    const int ctx = a.ctx_len[r];
    int lo = 0, hi = G - 1;  // the last group that starts at or before r (empty ones come first)
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (start[mid] <= r)
        lo = mid;
      else
        hi = mid - 1;
    }
    const int s0 = start[lo], prefix = a.prefix_len[lo];
    const bool wrong =
        prefix < 0 || prefix > cap || ctx < 0 || ctx > cap || (ctx > 0 && ctx < prefix);
    if (wrong) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
    const bool active = !wrong && ctx > 0;
    if (active) atomicMin(lead + lo, r);
    p.req_state[r] = !wrong;
    p.req_group[r] = active ? lo : -1;
    p.req_at[r] = r - s0;
    p.req_size[r] = start[lo + 1] - s0;
    p.req_prefix[r] = prefix;
  }
  __syncthreads();
  // groups: the blocks of each prefix. units and listed ones per class, counts packed
  long long base[2] = {0, 0};
  int listed[2] = {0, 0};
  for (int g0 = 0; g0 < G; g0 += kPlanThr) {
    const int g = g0 + tid;
    int s0 = 0, n = 0, prefix = 0, l = 0x7FFFFFFF, c = 0;
    long long units = 0;
    if (g < G) {
      s0 = start[g];
      n = start[g + 1] - s0;
      prefix = a.prefix_len[g];
      l = near_g ? near_lead[g] : __ldcg(p.lead + g);
      if (l != 0x7FFFFFFF && prefix > 0) {
        c = class_of(a.shape, n * hpk);
        const PrefixClass k = by_class(c, a.shape.cls[0], a.shape.cls[1]);
        units = (long long)a.n_kv * k.vh * ceil_div(n * hpk, k.rb) * tiles_of(0, prefix, k.tile_sh);
      }
    }
    const long long one = units > 0 ? 1ll << (32 * c) : 0;
    long long x[3] = {c == 0 ? units : 0, c == 1 ? units : 0, one}, total[3];
    plan_scan(x, total);
    if (g < G) {
      const long long at = by_class(c, base[0] + x[0], base[1] + x[1]) - units;
      if (units > 0) {
        const int k = by_class(c, listed[0], listed[1]) + (int)((x[2] - one) >> (32 * c));
        const PrefixPlan::Lists to = lists_of(p, c);
        to.g_u0[k] = at;
        if (c == 0 && k < kPlanNear) near_u0[k] = at;
        to.g_first[k] = s0;
        to.g_size[k] = n;
        to.g_prefix[k] = prefix;
        to.g_lead[k] = l;
      }
      p.gr_u0[g] = units > 0 ? at : -1;
    }
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      base[k] += total[k];
      listed[k] += (int)(total[2] >> (32 * k));
    }
  }
  __syncthreads();
  // requests: the blocks of their own tokens
  const long long prefix_units[2] = {base[0], base[1]};
  const PrefixClass ok = by_class(own_cls, a.shape.cls[0], a.shape.cls[1]);
  const int blocks = a.n_kv * ok.vh * ceil_div(hpk, ok.rb);
  int own_listed = 0;
  for (int r0 = 0; r0 < R; r0 += kPlanThr) {
    const int r = r0 + tid;
    const int g = r < R ? p.req_group[r] : -1;
    const int prefix = g >= 0 ? p.req_prefix[r] : 0, ctx = g >= 0 ? a.ctx_len[r] : 0;
    const long long units = (long long)blocks * tiles_of(prefix, ctx, ok.tile_sh);
    long long x[2] = {units, units > 0}, total[2];
    plan_scan(x, total);
    if (r < R) {
      const long long at = by_class(own_cls, base[0], base[1]) + x[0] - units;
      p.req_pu0[r] = g >= 0 ? p.gr_u0[g] : -1;
      p.req_ou0[r] = units > 0 ? at : -1;
      if (units > 0) {
        const int k = own_listed + (int)x[1] - 1;
        p.r_u0[k] = at;
        if (k < kPlanNear) near_r[k] = at;
        p.r_list[k] = r;
        p.r_from[k] = prefix;
        p.r_to[k] = ctx;
      }
    }
    base[0] += own_cls ? 0 : total[0];
    base[1] += own_cls ? total[0] : 0;
    own_listed += (int)total[1];
  }
  __syncthreads();
  // workers: with fewer units than would give each `least`, fewer have any
#pragma unroll 1
  for (int c = 0; c < 2; ++c) {
    const PrefixClass k = by_class(c, a.shape.cls[0], a.shape.cls[1]);
    const PrefixPlan::Lists list = lists_of(p, c);
    const long long U = c ? base[1] : base[0], own0 = c ? prefix_units[1] : prefix_units[0];
    const int groups = c ? listed[1] : listed[0];
    const long long few = div_pos(U + k.least - 1, k.least);
    int n = (int)(few < k.n ? few : k.n);
    if (n == 0) {
      if (tid == 0) p.head[8 * c + 4] = 0;
      continue;
    }
    const long long quot = div_pos(U, n), rem = U - quot * n;
    if (tid == 0) {
      long long *head = p.head + 8 * c;
      head[0] = U;
      head[1] = groups;
      head[2] = quot;
      head[3] = rem;
      head[4] = n;
      head[7] = own0;
      p.head[16] = own_listed;
    }
    if (c == 1) break;
    // Workers for each block, in proportion to its tiles? Where that costs none more tiles than
    // about what a part of a second block costs it.
    if (own0 == U && groups <= kPlanThr) {
      int tiles = 0, nrb = 0, per = 0;
      if (tid < groups) {
        tiles = tiles_of(0, list.g_prefix[tid], k.tile_sh);
        nrb = ceil_div(list.g_size[tid] * hpk, k.rb);
        per = (int)div_pos((long long)tiles * n, U);
        const long long most = per ? ceil_div(tiles, per) : tiles;
        const bool two = min(list.g_size[tid] * hpk, k.rb) > kOwnRows;
        if (per == 0 || most > quot + (two ? kOwnExtraTwo : kOwnExtraOne)) worst = 1;
      }
      long long x[1] = {(long long)a.n_kv * k.vh * nrb * per}, all[1];
      plan_scan(x, all);  // at most n: each is rounded down
      if (tid < groups) {
        near_w0[tid] = (int)(x[0] - (long long)a.n_kv * k.vh * nrb * per);
        near_k[tid] = per;
      }
      __syncthreads();
      if (!worst) {
        n = (int)all[0];
        for (int w = tid; w < n; w += kPlanThr) {
          int lo = 0, hi = groups - 1;
          while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (near_w0[mid] <= w)
              lo = mid;
            else
              hi = mid - 1;
          }
          const int to = list.g_prefix[lo], size = list.g_size[lo], per = near_k[lo];
          const int tiles = tiles_of(0, to, k.tile_sh), nrb = ceil_div(size * hpk, k.rb);
          const int b = (w - near_w0[lo]) / per, j = w - near_w0[lo] - b * per, kh = b / nrb;
          const int q = tiles / per, r = tiles - q * per, t = (int)first_unit(q, r, j);
          int4 *rec = list.start + 3 * w;
          rec[0] = make_int4(lo, b - kh * nrb, kh, t);
          rec[1] = make_int4(list.g_first[lo], size, list.g_lead[lo], 0);
          rec[2] = make_int4(to, (int)first_unit(q, r, j + 1) - t, per - 1 - j, 0);
        }
        if (tid == 0) p.head[4] = n;
        continue;
      }
    }
    for (int w = tid; w < n; w += kPlanThr) {
      const long long u = first_unit(quot, rem, w);
      const bool own = u >= own0;
      const int count = own ? own_listed : groups;
      const long long *u0 = count <= kPlanNear ? (own ? near_r : near_u0)
                                               : (own ? p.r_u0 : list.g_u0);
      int lo = 0, hi = count - 1;  // the last listed one that starts at or before u
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (u0[mid] <= u)
          lo = mid;
        else
          hi = mid - 1;
      }
      const int from = own ? p.r_from[lo] : 0, to = own ? p.r_to[lo] : list.g_prefix[lo];
      const int tiles = tiles_of(from, to, k.tile_sh);
      const int first = own ? p.r_list[lo] : list.g_first[lo];
      const int size = own ? 1 : list.g_size[lo], lead = own ? first : list.g_lead[lo];
      const int nrb = ceil_div(size * hpk, k.rb);
      const long long d = u - u0[lo], b = div_pos(d, tiles), kh = div_pos(b, nrb);
      int4 *rec = list.start + 3 * w;
      rec[0] = make_int4(lo | (own ? 1 << 30 : 0), (int)(b - kh * nrb), (int)kh,
                         (int)(d - b * tiles));
      rec[1] = make_int4(first, size, lead, from);
      rec[2] = make_int4(to, 0, -1, 0);
    }
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
constexpr int kTileSh = 8, kTile = 1 << kTileSh;
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
  const PrefixPlan plan = prefix_plan(a.shape, a.ws, a.n_reqs, a.hq, a.dv);
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
  ptx::launch_dependents();
  ptx::wait_for_previous();
  SegmentWalk<1> walk;
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
      segment_out<1>(a, plan, s, blockIdx.x, g, d == 0, &o, &lse);
      o[d] = l[g] == 0.f ? 0.f : sum / l[g];
      if (d == 0) *lse = l[g] == 0.f ? neg_inf : m[g] + logf(l[g]);
    }
  }
}

// ---------------------------------------------------------------------------------------
// Merge: one warp per (request, query head) and kCols columns. The parts of a row are its home
// places and the carries of the workers that start inside its blocks: the lanes take their
// log-sum-exps, then every lane adds up its columns of eight parts at a time. One rounding to
// bf16. Bound: the latency of a chain of loads (request, places, log-sum-exps, parts), then the
// bytes of the parts. Three CTAs an SM (80 registers), so that a call is one wave: with 99 and two
// CTAs 128 requests take 3 us more; with 64 registers spills cost as much.
// ---------------------------------------------------------------------------------------

constexpr int kCols = 128;  // columns of a warp: four a lane

__global__ void __launch_bounds__(kThr, 3) prefix_merge_kernel(const __grid_constant__ PrefixArgs a,
                                                               int slices) {
  const PrefixPlan p = prefix_plan(a.shape, a.ws, a.n_reqs, a.hq, a.dv);
  const int lane = threadIdx.x & 31;
  // fewer than 2^31 warps: 65535 requests x 256 heads x 8 slices
  const unsigned w = blockIdx.x * (kThr / 32) + (threadIdx.x >> 5);
  const unsigned n_rh = (unsigned)a.n_reqs * a.hq;
  if (w >= n_rh * slices) return;
  const unsigned rh = w / slices;
  const int col = (int)(w - rh * slices) * kCols, r = (int)(rh / (unsigned)a.hq);
  const float neg_inf = -__int_as_float(0x7f800000);
  ptx::wait_for_previous();
  const bool have[2] = {p.req_pu0[r] >= 0, p.req_ou0[r] >= 0};
  if (!p.req_state[r] | *a.gave_up) return;  // loaded together
  const int size = p.req_size[r];
  // the row's blocks: prefix, own part. Part 0 of a block is the home place, the rest are carries
  const float *home_o[2], *home_z[2], *carry_o[2], *carry_z[2];
  int parts[2] = {0, 0}, rb[2] = {0, 0}, dvh[2] = {0, 0};
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int c = class_of(a.shape, (b ? 1 : size) * a.hpk);
    const int vh = c ? a.shape.cls[1].vh : a.shape.cls[0].vh;
    rb[b] = c ? a.shape.cls[1].rb : a.shape.cls[0].rb;
    dvh[b] = vh == 2 ? a.dv >> 1 : a.dv;
    const int half = col >= dvh[b], off = col - half * dvh[b];
    const long long z = (b * 2ll + half) * n_rh + rh;
    home_o[b] = p.home_o + ((long long)b * n_rh + rh) * a.dv + col;
    home_z[b] = p.home_lse + z;
    if (have[b]) {
      const int2 more = p.home_more[z];
      parts[b] = 1 + more.y;
      carry_o[b] = (c ? p.cls[1].carry_o : p.cls[0].carry_o) + (long long)more.x * dvh[b] + off;
      carry_z[b] = (c ? p.cls[1].carry_lse : p.cls[0].carry_lse) + more.x;
    }
  }
  const int np = parts[0] + parts[1];
  auto block_of = [&](int i) { return i >= parts[0]; };
  auto lse_of = [&](int i) {
    const int b = block_of(i), k = b ? i - parts[0] : i;
    const float *z = b ? (k ? carry_z[1] : home_z[1]) : (k ? carry_z[0] : home_z[0]);
    return k ? z[(long long)(k - 1) * (b ? rb[1] : rb[0])] : *z;
  };
  float top = neg_inf;
  for (int i = lane; i < np; i += 32) top = fmaxf(top, lse_of(i));
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  const int mine = col + 4 * lane;
  const bool in = mine < a.dv;
  float sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i0 = 0; i0 < np; i0 += 32) {
    // a part of no mass is left out; a NaN goes on
    const float z = i0 + lane < np ? lse_of(i0 + lane) : neg_inf;
    const float wt = z == neg_inf ? 0.f : exp2_approx((z - top) * kLog2e);
    float s = wt;
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    sum += s;
    const int m = min(32, np - i0);
    for (int j0 = 0; j0 < m; j0 += 8) {
      float4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int i = i0 + j0 + j, b = block_of(i), k = b ? i - parts[0] : i;
        const float *o = b ? (k ? carry_o[1] : home_o[1]) : (k ? carry_o[0] : home_o[0]);
        if (k) o += (long long)(k - 1) * (b ? rb[1] * dvh[1] : rb[0] * dvh[0]);
        v[j] = in && j0 + j < m ? *reinterpret_cast<const float4 *>(o + 4 * lane)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float f = __shfl_sync(0xffffffffu, wt, (j0 + j) & 31);
        if (j0 + j < m && f != 0.f) {
          acc[0] = fmaf(f, v[j].x, acc[0]);
          acc[1] = fmaf(f, v[j].y, acc[1]);
          acc[2] = fmaf(f, v[j].z, acc[2]);
          acc[3] = fmaf(f, v[j].w, acc[3]);
        }
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  if (in) {
    uint2 v;
    v.x = pack_bf16(acc[0] * inv, acc[1] * inv);
    v.y = pack_bf16(acc[2] * inv, acc[3] * inv);
    *reinterpret_cast<uint2 *>(a.out + (long long)rh * a.dv + mine) = v;
  }
  if (lane == 0 && col == 0) a.lse[rh] = sum == 0.f ? neg_inf : top + logf(sum);
}

}  // namespace

PrefixShape prefix_shape(const DevLayout &l, int hq) {
  PrefixShape s;
  if (prefix_tc_layout(l)) {
    s.cls[0] = prefix_tc_class(l, hq);
    s.cls[1] = prefix_thin_class(l);
    // A wide tile costs the same for any number of rows up to 128, thin ones as many times 16 as
    // there are rows. Eight groups over 4000 tokens, 28/4 heads of 128, thin | wide, in us: 14 rows
    // 45 | 61, 28 rows 58 | 67, 35 rows 75 | 62, 56 rows 92 | 61. MLA: 32 rows 43 | 57, 64 rows
    // 63 | 53.
    s.wide_rows = 32;
  } else {
    s.cls[0] = {1, 1, 1, 7, 1};  // not used: no block is wide
    s.cls[1] = {kRows, 1, 2 * kSms, kTileSh, 1};
    s.wide_rows = 0x7FFFFFFF;
  }
  return s;
}

size_t prefix_workspace(const DevLayout &l, long long n_reqs, int hq, int dv) {
  return prefix_plan(prefix_shape(l, hq), nullptr, n_reqs, hq, dv).total;
}

// The limit of the wide kernel's waits, in ns. A test sets it to 0, with which a call gives up
// before it has begun, to see what a call that gave up leaves.
extern "C" unsigned long long kamera_prefix_wait_ns;
unsigned long long kamera_prefix_wait_ns = kPrefixWaitNs;

cudaError_t launch_prefix_attention(const PrefixArgs &args, cudaStream_t s) {
  PrefixArgs a = args;
  a.wait_ns = kamera_prefix_wait_ns;
  a.gave_up = prefix_plan(a.shape, a.ws, a.n_reqs, a.hq, a.dv).gave_up;
  // per device and kind of layout, each with the kernels it runs: what one kind cannot have is
  // nothing to the others
  static int configured[64][4] = {{0}};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const int kind = !prefix_tc_layout(a.lay) ? 0
                   : a.lay.kind == KAMERA_MLA ? 1
                                              : (a.lay.hd == 128 ? 2 : 3);
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev][kind]) {
      if (kind == 0) {
        e = cudaFuncSetAttribute(prefix_gen_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 gen_plan(1024, 1024).total);
      } else {
        e = prepare_prefix_tc(a.lay);
        if (e == cudaSuccess) e = prepare_prefix_thin(a.lay);
      }
      if (e != cudaSuccess) return e;
      configured[dev][kind] = 1;
    }
  }
  prefix_plan_kernel<<<1, kPlanThr, 0, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int hpk = a.hpk;
  if (kind != 0) {
    // blocks can be wide only where the largest group would be, thin only where one request is
    const bool wide = (long long)a.n_reqs * hpk > a.shape.wide_rows;
    if (wide) e = launch_prefix_tc(a, s);
    if (e == cudaSuccess && hpk <= a.shape.wide_rows) e = launch_prefix_thin(a, wide, s);
  } else {
    e = launch_early(prefix_gen_kernel, dim3(a.shape.cls[1].n), kThr, gen_plan(a.dk, a.dv).total, s,
                     a);
  }
  if (e != cudaSuccess) return e;
  const int slices = (a.dv + kCols - 1) / kCols;
  const long long warps = (long long)a.n_reqs * a.hq * slices;
  return launch_early(prefix_merge_kernel, dim3((unsigned)((warps + kThr / 32 - 1) / (kThr / 32))),
                      kThr, 0, s, a, slices);
}

}  // namespace kamera
