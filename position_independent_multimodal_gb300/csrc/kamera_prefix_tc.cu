// Attention over shared prefixes on the tensor cores: GQA with head_dim 64 or 128, MLA with a
// latent of 512 and a rope band of 64. One persistent CTA per SM works its share of tiles off
// (kamera_prefix.cuh); a tile is 128 tokens against a block's query rows.
//
//   S [128 rows x 128 tokens] = Q K^T           tcgen05, Q and K from shared memory
//   P = bf16(2^(c S - c m)),  c = |scale| log2 e  one thread per row, P back into TMEM over S
//   O [128 rows x dims] += P V                   tcgen05, P from TMEM, V from shared memory
//
// The running maximum m that P is taken against is raised only when a row's new maximum exceeds
// it by more than 8 / c (a factor of 256 in P, which bf16 and float32 hold without loss), and
// then O is rescaled in TMEM; after the first tiles that is rare. The row sums l take the
// float32 weights, so l and the log-sum-exp carry no bf16 rounding.
//
// Roles: warps 0-3 and 4-7 one query row per thread (softmax, rescaling, output), warps 8-11
// gather K and V rows through the page table (cp.async, 16 bytes each, zero-filled where a token
// has no slot) into a ring of stages, warp 12 issues the MMAs, warps 13-15 load Q.
//   GQA: two tiles of 128 query rows share each K and V tile; the MMAs of one run during the
//        softmax of the other.
//   MLA: one tile of 128 rows and half of V's columns a CTA (O takes 256 TMEM columns; all 512
//        would leave none for S), S of the next tile issued before P V of this one.
// Layout: every operand tile is 128 rows of 128 bytes (64 elements), swizzled in 128-byte rows;
// V is read MN-major, so its rows land unchanged too.
#include <mutex>

#include "kamera_prefix.cuh"
#include "kamera_ptx.cuh"

namespace kamera {

namespace {

constexpr int kThr = 512;
constexpr int kTok = 128;              // tokens per tile
constexpr int kRow = 128;              // query rows per MMA
constexpr int kChunk = kTok * 128;     // bytes of a 128 x 64 bf16 operand tile
constexpr int kSlots = 4;              // tiles whose slots are kept
constexpr int kMasks = 8;              // tiles whose token masks are kept
constexpr unsigned long long kWaitNs = 2000000000ull;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// DK, DV: 64-column chunks of K and of the CTA's V columns; QT: tiles of query rows; UC: chunks
// per ring stage; NST: ring stages.
template <int DK_, int DV_, int QT_, int UC_, int NST_>
struct Shape {
  static constexpr int DK = DK_, DV = DV_, QT = QT_, UC = UC_, NST = NST_;
  static constexpr int kStage = UC * kChunk;
  static constexpr int q = 0;
  static constexpr int ring = QT * DK * kChunk;
  static constexpr int slot = ring + NST * kStage;   // int [kSlots][kTok]
  static constexpr int mask = slot + kSlots * kTok * 4;  // uint32 [kMasks][4]
  static constexpr int bar = mask + kMasks * 16;
  // mbarriers
  static constexpr int full = 0, empty = NST, q_full = 2 * NST, q_empty = q_full + 1,
                       s_full = q_empty + 1, p_full = s_full + 2, pv_done = p_full + 2,
                       o_free = pv_done + 2, mk_full = o_free + 2, last = mk_full + kMasks,
                       n_bar = last + 1;
  static constexpr int misc = bar + n_bar * 8;  // TMEM address, give-up flag
  static constexpr int total = misc + 16;
  static constexpr uint32_t o_col = 256;        // O of tile t at o_col + t * 128
  static_assert(total <= 232448, "shared memory of one CTA");
  static_assert(DK % UC == 0 && DV % UC == 0, "whole stages");
};

using Gqa128 = Shape<2, 2, 2, 2, 5>;
using Gqa64 = Shape<1, 1, 2, 1, 12>;
using Mla512 = Shape<9, 4, 1, 1, 5>;

// Wait for a phase, giving up after kWaitNs or when another thread has (then the kernel runs to
// its end without waiting, and reports it).
__device__ __forceinline__ void wait(uint32_t bar, uint32_t parity, volatile uint32_t *gave_up) {
  if (ptx::mbar_try_wait(bar, parity)) return;
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar, parity)) {
    if (*gave_up) return;
    if (ptx::globaltimer() - t0 > kWaitNs) {
      *gave_up = 1;
      return;
    }
  }
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Number of the first stage of K tile i and V tile i in a segment of n tiles, in the order in
// which the MMAs read them: QT 2: K0 V0 K1 V1 ...; QT 1: K0 K1 V0 K2 V1 ... V(n-1).
template <class S>
__device__ __forceinline__ long long k_seq(int i) {
  constexpr int k = S::DK / S::UC, v = S::DV / S::UC;
  if (S::QT == 2) return (long long)i * (k + v);
  return i == 0 ? 0 : k + (long long)(i - 1) * (k + v);
}
template <class S>
__device__ __forceinline__ long long v_seq(int i, int n) {
  constexpr int k = S::DK / S::UC, v = S::DV / S::UC;
  if (S::QT == 2) return (long long)i * (k + v) + k;
  return k + (long long)i * (k + v) + (i == n - 1 ? 0 : k);
}

template <class S>
__global__ void __launch_bounds__(kThr, 1) prefix_tc_kernel(const __grid_constant__ PrefixArgs a) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = ptx::smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PrefixPlan plan = prefix_plan(a.ws, a.n_reqs, a.hq, a.dv, a.vh, a.rb, a.n_ctas);
  const DevLayout &lay = a.lay;
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + S::misc);
  volatile uint32_t *gave_up = misc + 1;
  auto bar = [&](int i) { return sb + S::bar + 8 * i; };

  if (sb & 1023u) {  // the swizzled layouts want 1024-byte groups; there is no static memory here
    if (tid == 0) atomicOr(a.status, KAMERA_DEVICE_TIMEOUT);
    return;
  }
  if (warp == 12) {
    ptx::tmem_alloc(sb + S::misc, 512);
    ptx::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < S::NST; ++i) {
      ptx::mbar_init(bar(S::full + i), 128);
      ptx::mbar_init(bar(S::empty + i), 1);
    }
    ptx::mbar_init(bar(S::q_full), 96);
    ptx::mbar_init(bar(S::q_empty), 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(S::s_full + i), 1);
      ptx::mbar_init(bar(S::p_full + i), 128);
      ptx::mbar_init(bar(S::pv_done + i), 1);
      ptx::mbar_init(bar(S::o_free + i), 128);
    }
    for (int i = 0; i < kMasks; ++i) ptx::mbar_init(bar(S::mk_full + i), 4);
    ptx::mbar_init(bar(S::last), 1);
    ptx::fence_mbar_init();
    *gave_up = 0;
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];

  SegmentWalk walk;
  walk.start(a, plan, blockIdx.x);
  Segment s;

  if (warp < 8) {
    // ---- softmax: thread = query row ----
    const int w = warp >> 2;                       // query tile (QT 1: only warps 0-3 work)
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const int row = (warp & 3) * 32 + lane;
    const float c = fabsf(a.scale) * kLog2e;
    const bool flip = a.scale < 0.f;
    const float neg_inf = -__int_as_float(0x7f800000);
    const uint32_t o_t = tmem + S::o_col + (S::QT == 2 ? w * 128 : 0) + lane_off;
    uint32_t used[2] = {0, 0};  // S buffers taken so far
    uint32_t tiles = 0;         // tiles of this query tile so far (phases of pv_done)
    uint32_t seen = 0;          // tiles the loader has masked so far
    while (walk.next(a, plan, &s)) {
      const int n = (s.tok1 - s.tok0 + kTok - 1) / kTok;
      if (S::QT == 2 ? (w == 1 && s.rows <= kRow) : w == 1) {
        seen += n;
        continue;
      }
      const bool live = kRow * w + (row & ~31) < s.rows;  // a warp without rows only keeps step
      float m = neg_inf, l = 0.f;
      for (int i = 0; i < n; ++i, ++seen, ++tiles) {
        const int b = S::QT == 2 ? w : (i & 1);
        wait(bar(S::s_full + b), used[b] & 1, gave_up);
        __syncwarp();
        ++used[b];
        ptx::tc_fence_after();
        if (live) {
          const uint32_t st = tmem + b * 128 + lane_off;
          const int mk = seen % kMasks;
          wait(bar(S::mk_full + mk), (seen / kMasks) & 1, gave_up);
          __syncwarp();
          const uint4 msk = *reinterpret_cast<const uint4 *>(smem + S::mask + 16 * mk);
          const bool whole = (msk.x & msk.y & msk.z & msk.w) == 0xffffffffu;
          float mx = m;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t r[32];
            ptx::tmem_ld32(st + 32 * j, r);
#pragma unroll
            for (int e = 0; e < 32; e += 8) ptx::tmem_ld_wait(r + e);
            if (!whole || flip) {
              const uint32_t bits = j == 0 ? msk.x : j == 1 ? msk.y : j == 2 ? msk.z : msk.w;
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float x = __uint_as_float(r[e]);
                mx = (bits >> e) & 1 ? fmaxf(mx, flip ? -x : x) : mx;
              }
            } else {
              float m0 = mx, m1 = mx, m2 = mx, m3 = mx;
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                m0 = fmaxf(m0, __uint_as_float(r[e]));
                m1 = fmaxf(m1, __uint_as_float(r[e + 1]));
                m2 = fmaxf(m2, __uint_as_float(r[e + 2]));
                m3 = fmaxf(m3, __uint_as_float(r[e + 3]));
              }
              mx = fmaxf(fmaxf(m0, m1), fmaxf(m2, m3));
            }
          }
          const bool first = m == neg_inf && mx > neg_inf;
          const bool raise = first || (mx - m) * c > 8.f;
          if (__any_sync(0xffffffffu, raise)) {
            const float f = raise ? (first ? 0.f : exp2_approx((m - mx) * c)) : 1.f;
            if (raise) m = mx;
            if (i > 0) {
              wait(bar(S::pv_done + (S::QT == 2 ? w : 0)), (tiles - 1) & 1, gave_up);
              __syncwarp();
              ptx::tc_fence_after();
              l *= f;
#pragma unroll 1
              for (int j = 0; j < S::DV * 2; ++j) {
                uint32_t r[32];
                ptx::tmem_ld32(o_t + 32 * j, r);
#pragma unroll
                for (int e = 0; e < 32; e += 8) ptx::tmem_ld_wait(r + e);
#pragma unroll
                for (int e = 0; e < 32; ++e) r[e] = __float_as_uint(__uint_as_float(r[e]) * f);
                ptx::tmem_st32(o_t + 32 * j, r);
              }
            }
          }
          const float base = m > neg_inf ? m * c : 0.f;
          const float cs = flip ? -c : c;
          float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t r[32];
            ptx::tmem_ld32(st + 32 * j, r);
#pragma unroll
            for (int e = 0; e < 32; e += 8) ptx::tmem_ld_wait(r + e);
            float p[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) p[e] = exp2_approx(fmaf(__uint_as_float(r[e]), cs, -base));
            if (!whole) {
              const uint32_t bits = j == 0 ? msk.x : j == 1 ? msk.y : j == 2 ? msk.z : msk.w;
#pragma unroll
              for (int e = 0; e < 32; ++e) p[e] = (bits >> e) & 1 ? p[e] : 0.f;
            }
            uint32_t h[16];
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              l0 += p[e];
              l1 += p[e + 1];
              l2 += p[e + 2];
              l3 += p[e + 3];
              h[e / 2] = pack_bf16(p[e], p[e + 1]);
              h[e / 2 + 1] = pack_bf16(p[e + 2], p[e + 3]);
            }
            ptx::tmem_st16(st + 16 * j, h);
          }
          l += (l0 + l1) + (l2 + l3);
          ptx::tmem_st_wait();
        }
        ptx::tc_fence_before();
        ptx::mbar_arrive(bar(S::p_full + b));
      }
      // S of a tile says that P V two (QT 1) or one (QT 2) tiles before it is complete, so a wait
      // for the next phase cannot mistake an older one for it; the last two are waited for in turn
      const uint32_t pv = bar(S::pv_done + (S::QT == 2 ? w : 0));
      if (S::QT == 1 && n > 1) wait(pv, (tiles - 2) & 1, gave_up);
      wait(pv, (tiles - 1) & 1, gave_up);
      __syncwarp();
      ptx::tc_fence_after();
      const int i = kRow * w + row;
      if (live) {
        float *o = nullptr, *lse = nullptr;
        if (i < s.rows) segment_out(a, plan, s, blockIdx.x, i, &o, &lse);
        const bool ok = l != 0.f && !*gave_up;
        const float inv = 1.f / l;
#pragma unroll 1
        for (int j = 0; j < S::DV * 2; ++j) {
          uint32_t r[32];
          ptx::tmem_ld32(o_t + 32 * j, r);
#pragma unroll
          for (int e = 0; e < 32; e += 8) ptx::tmem_ld_wait(r + e);
          if (o) {
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float4 v;
              v.x = ok ? __uint_as_float(r[e]) * inv : 0.f;
              v.y = ok ? __uint_as_float(r[e + 1]) * inv : 0.f;
              v.z = ok ? __uint_as_float(r[e + 2]) * inv : 0.f;
              v.w = ok ? __uint_as_float(r[e + 3]) * inv : 0.f;
              *reinterpret_cast<float4 *>(o + 32 * j + e) = v;
            }
          }
        }
        if (o) *lse = ok ? (m * c + log2f(l)) * kLn2 : neg_inf;
      }
      ptx::tc_fence_before();
      ptx::mbar_arrive(bar(S::o_free + w));
    }
  } else if (warp < 12) {
    // ---- K and V rows into the ring ----
    const int lt = tid - 256;
    const bool gqa = lay.kind == KAMERA_GQA;
    const long long layer_k = (long long)a.layer * a.pool.num_slots * lay.row_k;
    const long long layer_v = (long long)a.layer * a.pool.num_slots * lay.row_v;
    int *slots = reinterpret_cast<int *>(smem + S::slot);
    uint32_t *masks = reinterpret_cast<uint32_t *>(smem + S::mask);
    const int piece = lt & 7, t_lo = lt >> 3;  // 16-byte piece of a row, first token
    uint32_t seq = 0, tile_no = 0;             // stages and tiles so far
    while (walk.next(a, plan, &s)) {
      const int n = (s.tok1 - s.tok0 + kTok - 1) / kTok;
      const __nv_bfloat16 *kb = a.pool.k + layer_k + (gqa ? s.kvh * lay.hd : 0) + 8 * piece;
      const __nv_bfloat16 *vb = gqa ? a.pool.v + layer_v + s.kvh * lay.hd + 8 * piece
                                    : a.pool.k + layer_k + s.half * (S::DV * 64) + 8 * piece;
      const int vrow = gqa ? lay.row_v : lay.row_k;
      // `chunks` chunks of the tile whose slots are sl into the next stages
      auto issue = [&](const __nv_bfloat16 *src, int row, int chunks, const int *sl) {
        for (int u = 0; u < chunks / S::UC; ++u, ++seq) {
          const int st = seq % S::NST;
          wait(bar(S::empty + st), (seq / S::NST + 1) & 1, gave_up);
          const uint32_t dst = sb + S::ring + st * S::kStage;
#pragma unroll
          for (int j = 0; j < kTok / 16; ++j) {
            const int t = t_lo + 16 * j, slot = sl[t];
            const __nv_bfloat16 *p = slot >= 0 ? src + (long long)slot * row + u * S::UC * 64
                                               : a.pool.k;
#pragma unroll
            for (int k = 0; k < S::UC; ++k)
              ptx::cp_async16(dst + k * kChunk + t * 128 + ((piece ^ (t & 7)) << 4), p + k * 64,
                              slot >= 0 ? 16u : 0u);
          }
          ptx::cp_async_mbar_arrive(bar(S::full + st));
        }
      };
      auto load_k = [&](int i) {
        const long long tok = s.tok0 + (long long)i * kTok + lt;
        int slot = -1;
        if (tok < s.tok1) slot = (int)slot_of(a.pool, lay.page_size, s.lead, tok, a.status);
        const int k = tile_no % kSlots, mk = tile_no % kMasks;
        ++tile_no;
        slots[k * kTok + lt] = slot;
        const uint32_t bits = __ballot_sync(0xffffffffu, slot >= 0);
        if (lane == 0) {
          masks[4 * mk + (warp & 3)] = bits;
          ptx::mbar_arrive(bar(S::mk_full + mk));
        }
        __syncwarp();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        issue(kb, lay.row_k, S::DK, slots + k * kTok);
      };
      const uint32_t t0 = tile_no;
      auto load_v = [&](int i) {
        issue(vb, vrow, S::DV, slots + ((t0 + i) % kSlots) * kTok);
      };
      load_k(0);
      for (int i = 0; i < n; ++i) {
        if (S::QT == 1 && i + 1 < n) load_k(i + 1);
        load_v(i);
        if (S::QT == 2 && i + 1 < n) load_k(i + 1);
      }
    }
    ptx::cp_async_wait_all();
  } else if (warp == 12) {
    // ---- MMAs, one thread ----
    if (lane == 0) {
      const uint32_t id_s = ptx::idesc_bf16_f32(kRow, kTok);
      const uint32_t id_o = ptx::idesc_bf16_f32(kRow, S::UC * 64) | (1u << 16);  // V MN-major
      uint32_t base = 0;                 // stages of earlier segments
      uint32_t segs = 0, p_used[2] = {0, 0}, o_used[2] = {0, 0};
      while (walk.next(a, plan, &s)) {
        const int n = (s.tok1 - s.tok0 + kTok - 1) / kTok;
        const int qt = S::QT == 2 ? (s.rows > kRow ? 2 : 1) : 1;
        // S of query tile t (TMEM buffer b) against K tile i; `first`: the stages' first reader
        auto mma_s = [&](int t, int b, int i, bool first, bool last) {
          const uint32_t q = sb + S::q + t * S::DK * kChunk;
          for (int u = 0; u < S::DK / S::UC; ++u) {
            const uint32_t seq = base + (uint32_t)k_seq<S>(i) + u, st = seq % S::NST;
            if (first) {
              wait(bar(S::full + st), (seq / S::NST) & 1, gave_up);
              ptx::fence_proxy_async_smem();
            }
            const uint32_t k = sb + S::ring + st * S::kStage;
#pragma unroll
            for (int x = 0; x < S::UC * 4; ++x) {
              const uint32_t off = (x >> 2) * kChunk + (x & 3) * 32;
              ptx::mma_bf16(tmem + b * 128, ptx::smem_desc_sw128(q + u * S::UC * kChunk + off),
                            ptx::smem_desc_sw128(k + off), id_s, (u | x) ? 1u : 0u);
            }
            if (last) ptx::mma_commit(bar(S::empty + st));
          }
          ptx::mma_commit(bar(S::s_full + b));
        };
        auto mma_o = [&](int t, int b, int i, bool first, bool last) {
          wait(bar(S::p_full + b), p_used[b] & 1, gave_up);
          ++p_used[b];
          if (i == 0) {  // the last segment's output has been read
            if (o_used[t]) wait(bar(S::o_free + t), (o_used[t] - 1) & 1, gave_up);
            ++o_used[t];
          }
          ptx::tc_fence_after();
          for (int u = 0; u < S::DV / S::UC; ++u) {
            const uint32_t seq = base + (uint32_t)v_seq<S>(i, n) + u, st = seq % S::NST;
            if (first) {
              wait(bar(S::full + st), (seq / S::NST) & 1, gave_up);
              ptx::fence_proxy_async_smem();
            }
            const uint32_t v = sb + S::ring + st * S::kStage;
#pragma unroll
            for (int x = 0; x < kTok / 16; ++x)
              ptx::mma_bf16_ta(tmem + S::o_col + t * 128 + u * S::UC * 64, tmem + b * 128 + 8 * x,
                               ptx::smem_desc_sw128_mn(v + x * 2048, kChunk), id_o,
                               (i | x) ? 1u : 0u);
            if (last) ptx::mma_commit(bar(S::empty + st));
          }
          ptx::mma_commit(bar(S::pv_done + t));
        };
        wait(bar(S::q_full), segs & 1, gave_up);
        ++segs;
        ptx::fence_proxy_async_smem();
        ptx::tc_fence_after();
        if (S::QT == 2) {
          for (int t = 0; t < qt; ++t) mma_s(t, t, 0, t == 0, t == qt - 1);
          if (n == 1) ptx::mma_commit(bar(S::q_empty));
          for (int i = 0; i < n; ++i)
            for (int t = 0; t < qt; ++t) {
              mma_o(t, t, i, t == 0, t == qt - 1);
              if (i + 1 < n) {
                mma_s(t, t, i + 1, t == 0, t == qt - 1);
                if (i + 2 == n && t == qt - 1) ptx::mma_commit(bar(S::q_empty));
              }
            }
        } else {
          mma_s(0, 0, 0, true, true);
          if (n == 1) ptx::mma_commit(bar(S::q_empty));
          for (int i = 0; i < n; ++i) {
            if (i + 1 < n) {
              mma_s(0, (i + 1) & 1, i + 1, true, true);
              if (i + 2 == n) ptx::mma_commit(bar(S::q_empty));
            }
            mma_o(0, i & 1, i, true, true);
          }
        }
        base += n * ((S::DK + S::DV) / S::UC);
      }
      ptx::mma_commit(bar(S::last));  // no MMA is in flight when the TMEM goes back
      if (!ptx::mbar_wait(bar(S::last), 0, kWaitNs)) *gave_up = 1;
    }
    __syncwarp();
  } else {
    // ---- Q ----
    const int lt = tid - 13 * 32;
    uint32_t segs = 0;
    while (walk.next(a, plan, &s)) {
      if (segs) wait(bar(S::q_empty), (segs - 1) & 1, gave_up);
      ++segs;
      const int rows = s.rows > kRow ? 2 * kRow : kRow;
      for (int e = lt; e < rows * S::DK * 8; e += 96) {
        const int piece = e & 7, x = e >> 3, ch = x % S::DK, i = x / S::DK;
        const uint32_t dst = sb + S::q + ((i >> 7) * S::DK + ch) * kChunk + (i & 127) * 128 +
                             ((piece ^ (i & 7)) << 4);
        const __nv_bfloat16 *src = a.q;
        if (i < s.rows) {
          int r, h;
          segment_row(a, s, i, &r, &h);
          src += ((long long)r * a.hq + h) * a.dk + ch * 64 + piece * 8;
        }
        ptx::cp_async16(dst, src, i < s.rows ? 16u : 0u);
      }
      ptx::cp_async_mbar_arrive(bar(S::q_full));
    }
    ptx::cp_async_wait_all();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (tid == 0 && *gave_up) atomicOr(a.status, KAMERA_DEVICE_TIMEOUT);
  if (warp == 12) ptx::tmem_dealloc(tmem, 512);
}

template <class S>
cudaError_t configure() {
  return cudaFuncSetAttribute(prefix_tc_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              S::total);
}

template <class S>
cudaError_t launch(const PrefixArgs &a, cudaStream_t s) {
  prefix_tc_kernel<S><<<a.n_ctas, kThr, S::total, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

bool prefix_tc_layout(const DevLayout &l) {
  return (l.kind == KAMERA_GQA && (l.hd == 64 || l.hd == 128)) ||
         (l.kind == KAMERA_MLA && l.latent == 512 && l.rope_d == 64);
}

void prefix_tc_shape(const DevLayout &l, int *rb, int *tile, int *vh, int *n_ctas) {
  const bool gqa = l.kind == KAMERA_GQA;
  *rb = gqa ? 2 * kRow : kRow;
  *tile = kTok;
  *vh = gqa ? 1 : 2;
  *n_ctas = kPrefixCtas;
}

cudaError_t prepare_prefix_tc() {
  cudaError_t e = configure<Gqa128>();
  if (e == cudaSuccess) e = configure<Gqa64>();
  if (e == cudaSuccess) e = configure<Mla512>();
  return e;
}

cudaError_t launch_prefix_tc(const PrefixArgs &a, cudaStream_t s) {
  if (a.lay.kind == KAMERA_MLA) return launch<Mla512>(a, s);
  return a.lay.hd == 128 ? launch<Gqa128>(a, s) : launch<Gqa64>(a, s);
}

}  // namespace kamera
