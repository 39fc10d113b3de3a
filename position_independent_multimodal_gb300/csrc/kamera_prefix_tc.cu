// Wide blocks of attention over shared prefixes, on the tensor cores: GQA with head_dim 64 or
// 128, MLA with a latent of 512 and a rope band of 64. One persistent CTA per SM works its share
// of tiles off (kamera_prefix.cuh); a tile is 128 tokens against a block's query rows.
//
//   S [128 rows x 128 tokens] = Q K^T           tcgen05, Q and K from shared memory
//   P = bf16(2^(c S - c m)),  c = |scale| log2 e  two threads per row, P into TMEM over S
//   O [128 rows x dims] += P V                   tcgen05, P from TMEM, V from shared memory
//
// The running maximum m that P is taken against is raised only when a row's new maximum exceeds
// it by more than 8 / c (a factor of 256 in P, which bf16 and float32 hold without loss), and
// then O is rescaled in TMEM; after the first tiles that is rare. The row sums l take the
// float32 weights, so l and the log-sum-exp carry no bf16 rounding.
//
// P is rounded to bf16, the one rounding between the scores and the output's own: both operands of
// a product have one type, and V is bf16. It moves an output by at most 2^-8 sum p|V| / l, the size
// of the output's own rounding; over many tokens the errors' signs differ and their mean falls with
// the square root of their number (against float64 the listed cases are 1.2 to 1.4 times as far off
// as float32 weights rounded once at the end). Float32 weights would take V converted to tf32,
// twice its bytes of shared memory and half the rate, or P in two bf16 terms, PV's products twice;
// layouts on the CUDA cores keep them.
//
// Roles: warps 0-15 (MLA 0-7) softmax, rescaling and output, two threads (of two warps) to a query
// row, 64 tokens and half of O's columns each; the next four bring K and V rows through the page
// table into a ring of stages; one thread of the next issues the MMAs and the copies of Q. Whole
// tiles of pages of 8, 16, 32 or 64 slots, or a multiple of 128, come as tensor-map copies, one
// per page and 64 columns; tiles with tokens left out (the ends of a context, pages outside the
// pool) and other page sizes as 16-byte cp.async, zero-filled where a token has no slot, so that
// nothing of a row that no token holds is ever multiplied.
//   GQA: two tiles of 128 query rows share each K and V tile; the MMAs of one run during the
//        softmax of the other. O and S of both fill the TMEM, so S of a tile waits for P V of the
//        tile before: the chain S (512 cycles), softmax, P V (512) of a query tile is what bounds
//        it. The softmax therefore takes its weights against the maximum so far, in one pass over
//        S, and finds the tile's maximum on the way; only when that raises m are they taken again.
//        3200 cycles a pair of tiles, of which the tensor core works 2050 (2 x 4 x 256): 101 us
//        for 896 rows on 4 KV heads over 65500 tokens, 1.19 PFLOP/s, 61 % of a large library
//        product. Tried and slower: S of 64 tokens in two buffers (an MMA of N = 64 takes as long
//        as one of N = 128), one thread to a row, two loading warps (a thread issues a 2 KB copy
//        in about 107 cycles: 700 of 3500 cycles waiting for K and V).
//   MLA: one tile of 128 rows and half of V's columns a CTA (O takes 256 TMEM columns; all 512
//        would leave none for S), S of the next tile issued before P V of this one. 144 KB of Q
//        leave a ring of 80 KB, whose latency bounds it (9000 cycles a tile, 4400 of them MMAs):
//        41 us for 40 x 16 rows over two prefixes of 9003 tokens.
// Layout: every operand tile is 128 rows of 128 bytes (64 elements), swizzled in 128-byte rows;
// V is read MN-major, so its rows land unchanged too.
#include "kamera_prefix.cuh"
#include "kamera_ptx.cuh"
#include "kamera_smem.cuh"
#include "kamera_tc.cuh"

namespace kamera {

namespace {

constexpr int kTokSh = 7, kTok = 1 << kTokSh;  // tokens per tile
constexpr int kRow = 128;              // query rows per MMA
constexpr int kMasks = 8;              // tiles whose token masks are kept

// DK, DV: 64-column chunks of K and of the CTA's V columns; QT: tiles of query rows; UC: chunks
// per ring stage; NST: ring stages; NL: warps that load K and V.
template <int DK_, int DV_, int QT_, int UC_, int NST_, int NL_>
struct Shape {
  static constexpr int DK = DK_, DV = DV_, QT = QT_, UC = UC_, NST = NST_, NL = NL_;
  static constexpr int kSoft = 8 * QT, kMma = kSoft + NL;  // softmax warps; the MMA warp
  // With two query tiles the softmax warps take registers of the others; whole warpgroups. The
  // kernel is compiled under the cap of its threads all the same (80 registers a thread for 768):
  // GQA 128 spills 412 bytes and loads 332, GQA 64 400 and 328; MLA (128 registers) 84 and 64
  static constexpr bool kShift = QT == 2;
  static constexpr int kThr = 32 * (kShift ? (kMma + 4) / 4 * 4 : kMma + 1);
  static constexpr int kRegsSoft = 96, kRegsRest = 48;
  static constexpr int kRegs = 32 * kSoft * kRegsSoft + (kThr - 32 * kSoft) * kRegsRest;
  static constexpr int kStage = UC * kChunk;
  static constexpr int q = 0;
  // the queries' place takes the output on its way out, 4 KB a softmax warp
  static constexpr int ring = QT * DK * kChunk > kSoft * 4096 ? QT * DK * kChunk : kSoft * 4096;
  static constexpr int mask = ring + NST * kStage;  // uint32 [kMasks][4]
  static constexpr int xch = mask + kMasks * 16;    // float [2][2][kRow]: maxima, then sums
  static constexpr int bar = xch + 4 * kRow * 4;
  // mbarriers; those of P: [buffer][half of the tokens]
  static constexpr int full = 0, empty = NST, q_full = empty + NST, q_empty = q_full + 1,
                       s_full = q_empty + 1, p_full = s_full + 2, pv_done = p_full + 4,
                       o_free = pv_done + 2, o_full = o_free + 2,
                       mk_full = o_full + 2, last = mk_full + kMasks, n_bar = last + 1;
  static constexpr int misc = bar + n_bar * 8;  // TMEM address, give-up flag
  static constexpr int total = misc + 16;
  static constexpr uint32_t o_col = 256;        // O of tile t at o_col + t * 128
  static_assert(total <= 232448, "shared memory of one CTA");
  static_assert(DK % UC == 0 && DV % UC == 0, "whole stages");
};

using Gqa128 = Shape<2, 2, 2, 2, 5, 4>;
using Gqa64 = Shape<1, 1, 2, 1, 10, 4>;
using Mla512 = Shape<9, 4, 1, 1, 5, 4>;

// Tensor maps of a call: pool rows of the layer (boxes of 64 columns and `box` slots) and query
// rows (64 columns; a block of a group's rows, or one request's).
struct Maps {
  CUtensorMap k, v, q_group, q_own;
  int box;                    // slots per copy; 0: rows come by cp.async
  int q_step;                 // 1: the rows of a block are consecutive rows of q
  int group_bytes, own_bytes; // of the query copies
};

template <class S>
__global__ void __launch_bounds__(S::kThr, 1) prefix_tc_kernel(
    const __grid_constant__ PrefixArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = ptx::smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const PrefixPlan plan = prefix_plan(a.shape, a.ws, a.n_reqs, a.hq, a.dv);
  const DevLayout &lay = a.lay;
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + S::misc);
  volatile uint32_t *gave_up = misc + 1;
  auto bar = [&](int i) { return sb + S::bar + 8 * i; };
  // Waits for a phase, giving up after a.wait_ns or when another thread has. A thread that gave up
  // runs on to its end without waiting, arriving, copying or multiplying: it keeps step with the
  // named barriers only, and no barrier gets an arrival that it does not expect. Nothing of the
  // call's outputs is written then.
  bool dead = false;
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (dead || ptx::mbar_try_wait(b, parity)) return;
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait(b, parity)) {
      if (*gave_up || ptx::globaltimer() - t0 > a.wait_ns) {
        *gave_up = 1;
        dead = true;
        return;
      }
    }
  };
  auto arrive = [&](uint32_t b) {
    if (!dead) ptx::mbar_arrive(b);
  };

  // The swizzled layouts want 1024-byte groups (there is no static memory here, so they get them);
  // without them, or without time to wait, nothing is begun and the kernel ends as if it gave up.
  const bool begins = (sb & 1023u) == 0 && a.wait_ns != 0;
  if (warp == S::kMma) {
    ptx::tmem_alloc(sb + S::misc, 512);
    ptx::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < S::NST; ++i) {
      ptx::mbar_init(bar(S::full + i), 32 * S::NL);
      ptx::mbar_init(bar(S::empty + i), 1);
    }
    ptx::mbar_init(bar(S::q_full), 1);
    ptx::mbar_init(bar(S::q_empty), 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(S::s_full + i), 1);
      ptx::mbar_init(bar(S::p_full + 2 * i), 128);
      ptx::mbar_init(bar(S::p_full + 2 * i + 1), 128);
      ptx::mbar_init(bar(S::pv_done + i), 1);
      ptx::mbar_init(bar(S::o_free + i), 256);
      ptx::mbar_init(bar(S::o_full + i), 1);
    }
    for (int i = 0; i < kMasks; ++i) ptx::mbar_init(bar(S::mk_full + i), S::NL);
    ptx::mbar_init(bar(S::last), 1);
    ptx::fence_mbar_init();
    *gave_up = !begins;
    ptx::prefetch_map(&maps.k);
    ptx::prefetch_map(&maps.v);
    ptx::prefetch_map(&maps.q_group);
    ptx::prefetch_map(&maps.q_own);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];

  ptx::wait_for_previous();  // the plan
  ptx::launch_dependents();  // who starts from here on finds the plan complete
  SegmentWalk<0> walk;
  walk.start(a, plan, blockIdx.x);
  // the segment that follows is looked up while this one's first copies are on their way
  Segment s, after;
  bool more = begins && walk.next(a, plan, &after);

  if (warp < S::kSoft) {
    // ---- softmax: thread = half of a query row ----
    if (S::kShift) ptx::regs_more<S::kRegsSoft>();
    const int w = warp >> 3;                       // query tile
    const int hf = (warp >> 2) & 1;                // half of the tokens, of O's columns
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const float c = fabsf(a.scale) * kLog2e;
    const bool flip = a.scale < 0.f;
    const float neg_inf = -__int_as_float(0x7f800000);
    const uint32_t o_t = tmem + S::o_col + w * 128 + hf * (S::DV * 32) + lane_off;
    const uint32_t pv = bar(S::pv_done + w);
    float *xch = reinterpret_cast<float *>(smem + S::xch);
    const int pair = 2 + w * 4 + (warp & 3);  // named barrier of a row's two warps
    uint32_t s_ph = 0;   // parity of each S buffer
    uint32_t o_ph = 0;   // parity of o_full
    uint32_t tiles = 0;  // tiles of this query tile so far (phases of pv_done)
    uint32_t seen = 0;   // tiles the loader has masked so far
    while (more) {
      s = after;
      more = walk.next(a, plan, &after);
      const int n = tiles_of(s.tok0, s.tok1, kTokSh);
      if (w == 1 && s.rows <= kRow) {
        seen += n;
        continue;
      }
      const bool live = kRow * w + (row & ~31) < s.rows;  // a warp without rows only keeps step
      float m = neg_inf, l = 0.f;
      uint2 msk = make_uint2(0, 0);
      auto read_mask = [&]() {
        const int mk = seen % kMasks;
        wait(bar(S::mk_full) + 8 * mk, (seen / kMasks) & 1);
        __syncwarp();
        msk = *reinterpret_cast<const uint2 *>(smem + S::mask + 16 * mk + 8 * hf);
      };
      for (int i = 0; i < n; ++i, ++seen, ++tiles) {
        // the tile's mask. It is there before S is; of a segment's first tile it is read after
        // S, as this thread may be more tiles ahead of the loader than masks are kept
        if (live && i > 0) read_mask();
        const int b = S::QT == 2 ? w : (tiles & 1);
        wait(bar(S::s_full) + 8 * b, (s_ph >> b) & 1);
        __syncwarp();
        s_ph ^= 1u << b;
        ptx::tc_fence_after();
        if (live) {
          const uint32_t st = tmem + b * 128 + hf * 64 + lane_off;
          uint32_t x[32];
          ptx::tmem_ld32(st, x);
          if (i == 0) read_mask();
          const bool whole = (msk.x & msk.y) == 0xffffffffu;
          const float cs = flip ? -c : c;
          const f32x2 c2 = f2(cs, cs);
          float base = m > neg_inf ? m * c : 0.f;
          f32x2 la, lb;
          uint32_t h[32];
          float top = neg_inf, top2 = neg_inf;
          // the weights against `base`, their sums in la and lb, the maximum on the way; 32 columns
          // of S at a time, the first already on their way into x. Two copies of the loop: a test
          // of the mask at each weight would cost as much as the weight
          auto weights = [&](auto masked) {
            const f32x2 nb2 = f2(-base, -base);
            la = lb = f2(0.f, 0.f);
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              if (g) ptx::tmem_ld32(st + 32, x);
              ptx::tmem_ld_wait_all<32>(x);
              const uint32_t bits = g ? msk.y : msk.x;
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float y0 = __uint_as_float(x[e]), y1 = __uint_as_float(x[e + 1]);
                float p0, p1;
                f2_split(fma2(f2(y0, y1), c2, nb2), p0, p1);
                p0 = exp2_approx(p0);
                p1 = exp2_approx(p1);
                if (masked.v) {
                  const bool in0 = (bits >> e) & 1, in1 = (bits >> (e + 1)) & 1;
                  p0 = in0 ? p0 : 0.f;
                  p1 = in1 ? p1 : 0.f;
                  top = in0 ? fmaxf(top, flip ? -y0 : y0) : top;
                  top = in1 ? fmaxf(top, flip ? -y1 : y1) : top;
                } else {
                  float &t = e & 2 ? top2 : top;
                  t = fmaxf(fmaxf(t, y0), y1);
                }
                if (e & 2)
                  lb = add2(lb, f2(p0, p1));
                else
                  la = add2(la, f2(p0, p1));
                h[16 * g + e / 2] = pack_bf16(p0, p1);
              }
            }
            top = fmaxf(top, top2);
          };
          if (whole && !flip)
            weights(Int<0>());
          else
            weights(Int<1>());
          // the weights stand unless the maximum is to be raised, for either half of the row
          if (ptx::barrier_or(pair, 64,
                              (m == neg_inf && top > neg_inf) || (top - m) * c > 8.f)) {
            float *mine = xch + ((b * 2 + hf) << 7) + row;
            *mine = top;
            ptx::barrier_sync(pair, 64);
            top = fmaxf(top, xch[((b * 2 + (hf ^ 1)) << 7) + row]);
            const bool first = m == neg_inf && top > neg_inf;
            const bool raise = first || (top - m) * c > 8.f;
            const float f = raise ? (first ? 0.f : exp2_approx((m - top) * c)) : 1.f;
            if (raise) m = top;
            if (i > 0) {
              // P V of the tile before; that of the one before it is complete (this tile's S
              // says so) and this tile's waits for this thread, so the parity is unambiguous
              wait(pv, (tiles - 1) & 1);
              __syncwarp();
              ptx::tc_fence_after();
              l *= f;
#pragma unroll 1
              for (int j = 0; j < S::DV * 2; ++j) {
                uint32_t y[16];
                ptx::tmem_ld16(o_t + 16 * j, y);
                ptx::tmem_ld_wait_all<16>(y);
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                ptx::tmem_st16(o_t + 16 * j, y);
              }
              // The products of either half's tokens go into all of O's columns (GQA), and those
              // of the first half start on that half's arrival alone. So neither thread arrives
              // before both have scaled their columns.
              ptx::tmem_st_wait();
              ptx::tc_fence_before();
              ptx::barrier_sync(pair, 64);
              ptx::tc_fence_after();
            }
            base = m > neg_inf ? m * c : 0.f;
            ptx::tmem_ld32(st, x);
            weights(Int<1>());
          }
          ptx::tmem_st32(st + 32, h);  // P over the end of its half of S
          float l0, l1;
          f2_split(add2(la, lb), l0, l1);
          l += l0 + l1;
          ptx::tmem_st_wait();
        }
        ptx::tc_fence_before();
        arrive(bar(S::p_full) + 16 * b + 8 * hf);
      }
      wait(bar(S::o_full + w), o_ph);
      o_ph ^= 1;
      __syncwarp();
      ptx::tc_fence_after();
      if (live) {
        xch[((w * 2 + hf) << 7) + row] = l;
        ptx::barrier_sync(pair, 64);
        l += xch[((w * 2 + (hf ^ 1)) << 7) + row];
        ptx::barrier_sync(pair, 64);  // read before the next segment writes
        const int i = kRow * w + row;
        float *o = nullptr, *lse = nullptr;
        if (i < s.rows) segment_out<0>(a, plan, s, blockIdx.x, i, hf == 0, &o, &lse);
        const bool ok = l != 0.f && !*gave_up;
        const float inv = 1.f / l;
        // 32 columns at a time through shared memory (the queries are no longer needed), swizzled
        // in 16-byte pieces, so that a warp writes four whole lines of 128 bytes at a time
        uint4 *stage = reinterpret_cast<uint4 *>(smem + S::q + warp * 4096);
        const int piece = lane & 7;
#pragma unroll 1
        for (int j = 0; j < S::DV; ++j) {
          uint32_t r[32];
          ptx::tmem_ld32(o_t + 32 * j, r);
          ptx::tmem_ld_wait_all<32>(r);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            r[e] = ok ? __float_as_uint(__uint_as_float(r[e]) * inv) : 0u;
          __syncwarp();  // the columns before have been read
#pragma unroll
          for (int e = 0; e < 8; ++e)
            stage[8 * lane + (e ^ piece)] =
                make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int q = 4 * k + (lane >> 3);  // the row
            float *to = reinterpret_cast<float *>(
                __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(o), q));
            const uint4 v = stage[8 * q + (piece ^ (q & 7))];
            if (to) *reinterpret_cast<uint4 *>(to + hf * (S::DV * 32) + 32 * j + 4 * piece) = v;
          }
        }
        ptx::fence_proxy_async_smem();  // before the next queries are copied there
        if (o && hf == 0) *lse = ok ? (m * c + log2f(l)) * kLn2 : neg_inf;
      }
      ptx::tc_fence_before();
      arrive(bar(S::o_free + w));
    }
  } else if (warp < S::kMma) {
    if (S::kShift) ptx::regs_fewer<S::kRegsRest>();
    // ---- K and V rows into the ring: a warp brings kPart tokens of each tile, a lane holds the
    // slots of kLane. Copies by tensor map are issued by one thread of the warp, which stands in
    // for the others' arrivals; one issues a copy in about 100 cycles ----
    constexpr int kPart = kTok / S::NL, kLane = kPart / 32;
    const int part = warp - S::kSoft, t0 = kPart * part + lane;
    const bool gqa = lay.kind == KAMERA_GQA;
    const __nv_bfloat16 *lk = a.pool.k + (long long)a.layer * a.pool.num_slots * lay.row_k;
    const __nv_bfloat16 *lv =
        gqa ? a.pool.v + (long long)a.layer * a.pool.num_slots * lay.row_v : lk;
    const int vrow = gqa ? lay.row_v : lay.row_k;
    uint32_t *masks = reinterpret_cast<uint32_t *>(smem + S::mask);
    const int piece = lane & 7;  // cp.async: 16-byte piece of a row
    const int box = maps.box;    // slots of a copy; boxes: copies of this warp per 64 columns
    const int boxes = box == 0 ? 0 : (box <= kPart ? kPart / box : kPart * part % box == 0);
    struct Slots {
      int at[kLane];
      bool whole;  // every token of the tile is in
    };
    Place<S::NST> at;            // the next stage
    uint32_t tile_no = 0;        // tiles so far
    while (more) {
      s = after;
      const int n = tiles_of(s.tok0, s.tok1, kTokSh), a0 = s.tok0 / kTok;
      const int kcol = gqa ? s.kvh * lay.hd : 0;
      const int vcol = gqa ? kcol : s.half * (S::DV * 64);
      auto token = [&](int i, int k) {  // below 2^31: the tile starts below it
        const int tok = (a0 + i) * kTok + t0 + 32 * k;
        return tok >= s.tok0 && tok < s.tok1 ? tok : -1;
      };
      int page[kLane];  // of the next tile, not looked at yet
      auto load_pages = [&](int i) {
#pragma unroll
        for (int k = 0; k < kLane; ++k) {
          const int tok = token(i, k);
          page[k] = tok >= 0 ? load_page(a, s.lead, tok) : 0;
        }
      };
      // The next stages: `chunks` chunks from column `col` of a tile's rows
      auto issue = [&](const void *map, const __nv_bfloat16 *rows, int row, int col, int chunks,
                       const Slots &sl) {
        if (box && sl.whole) {
          int y[kPart / 8];  // first slots of the copies
#pragma unroll
          for (int k = 0; k < kPart / 8; ++k) {
            const int q = k * box;
            y[k] = __shfl_sync(0xffffffffu, q < 32 ? sl.at[0] : sl.at[kLane - 1], q & 31);
          }
          if (ptx::elect_one()) {
            Place<S::NST> to = at;
            for (int u = 0; u < chunks / S::UC; ++u) {
              const uint32_t full = bar(S::full) + 8 * to.st;
              uint32_t dst = sb + S::ring + to.st * S::kStage + kPart * part * 128;
              wait(bar(S::empty) + 8 * to.st, to.ph ^ 1);
              if (dead) break;
              if (boxes) {
                ptx::mbar_arrive_n(full, 31);
                ptx::mbar_arrive_expect_tx(full, boxes * box * S::UC * 128);
#pragma unroll
                for (int k = 0; k < kPart / 8; ++k) {
                  if (k < boxes) {
#pragma unroll
                    for (int c = 0; c < S::UC; ++c)
                      ptx::tma_2d(dst + c * kChunk, map, col + (u * S::UC + c) * 64, y[k], full);
                    dst += box * 128;
                  }
                }
              } else {
                ptx::mbar_arrive_n(full, 32);
              }
              to.advance(1);
            }
          }
          __syncwarp();
          at.advance(chunks / S::UC);
          return;
        }
        for (int u = 0; u < chunks / S::UC; ++u) {
          const uint32_t dst = sb + S::ring + at.st * S::kStage, full = bar(S::full) + 8 * at.st;
          wait(bar(S::empty) + 8 * at.st, at.ph ^ 1);
          at.advance(1);
          if (__any_sync(0xffffffffu, dead)) {
            dead = true;
            continue;
          }
          const __nv_bfloat16 *src = rows + col + u * S::UC * 64 + 8 * piece;
#pragma unroll 4
          for (int j = 0; j < kPart / 4; ++j) {  // four of this warp's tokens at a time
            const int q = 4 * j + (lane >> 3), t = kPart * part + q;
            const int slot = __shfl_sync(0xffffffffu, j < 8 ? sl.at[0] : sl.at[kLane - 1], q & 31);
            const __nv_bfloat16 *p = slot >= 0 ? src + (long long)slot * row : a.pool.k;
#pragma unroll
            for (int k = 0; k < S::UC; ++k)
              ptx::cp_async16(dst + k * kChunk + t * 128 + ((piece ^ (t & 7)) << 4),
                              slot >= 0 ? p + k * 64 : p, slot >= 0 ? 16u : 0u);
          }
          ptx::cp_async_mbar_arrive(full);
        }
      };
      Slots kt;  // of the last K tile
      auto load_k = [&](int i) {
        const int mk = tile_no++ % kMasks;
        uint32_t bits[kLane];
#pragma unroll
        for (int k = 0; k < kLane; ++k) {
          const int tok = token(i, k);
          kt.at[k] = tok >= 0 ? slot_in(a, page[k], tok) : -1;
          bits[k] = __ballot_sync(0xffffffffu, kt.at[k] >= 0);
        }
        if (i + 1 < n) load_pages(i + 1);  // ahead of its use
        if (lane == 0) {
#pragma unroll
          for (int k = 0; k < kLane; ++k) masks[4 * mk + part * kLane + k] = bits[k];
          arrive(bar(S::mk_full) + 8 * mk);
        }
        __syncwarp();
        ptx::barrier_sync(1, 32 * S::NL);
        const uint4 m = *reinterpret_cast<const uint4 *>(masks + 4 * mk);
        kt.whole = (m.x & m.y & m.z & m.w) == 0xffffffffu;
        issue(&maps.k, lk, lay.row_k, kcol, S::DK, kt);
      };
      load_pages(0);
      load_k(0);
      more = walk.next(a, plan, &after);
      for (int i = 0; i < n; ++i) {
        const Slots vt = kt;  // V of this tile may come after K of the next
        if (S::QT == 1 && i + 1 < n) load_k(i + 1);
        issue(&maps.v, lv, vrow, vcol, S::DV, vt);
        if (S::QT == 2 && i + 1 < n) load_k(i + 1);
      }
    }
    ptx::cp_async_wait_all();
  } else {
    if (S::kShift) ptx::regs_fewer<S::kRegsRest>();
    // ---- MMAs and Q, one thread. QT 2: S and P V of the two query tiles
    // in turn, so that the tensor core works on one during the softmax of the other; QT 1: S of a
    // tile before P V of the one before it. Issuing an MMA takes a few instructions only: the
    // descriptors of a tile's steps differ by constants ----
    if (warp == S::kMma && ptx::elect_one()) {
      // Q of a segment, once S of the one before is complete and its output has gone through Q's
      // place. Rows of a copy past the block's are other requests' or zero: their results go
      // nowhere
      uint32_t segs = 0, o_ph = 0;  // o_ph: a bit for each query tile
      bool two = false;             // the last segment had both
      auto load_q = [&]() {
        if (segs) {
          wait(bar(S::q_empty), (segs - 1) & 1);
          for (int t = 0; t <= two; ++t) {
            wait(bar(S::o_free + t), (o_ph >> t) & 1);
            o_ph ^= 1u << t;
          }
        }
        ++segs;
        two = S::QT == 2 && s.rows > kRow;
        if (dead) return;
        ptx::mbar_arrive_expect_tx(bar(S::q_full), s.own ? maps.own_bytes : maps.group_bytes);
        const int y = maps.q_step ? 0 : s.kvh * a.hpk;
        const int z = maps.q_step ? s.r0 * a.hq + s.row0 : s.r0 + s.row0 / a.hpk;
        for (int c = 0; c < S::DK; ++c)
          ptx::tma_3d(sb + S::q + c * S::QT * kChunk, s.own ? &maps.q_own : &maps.q_group, c * 64,
                      y, z, bar(S::q_full));
      };
      constexpr uint32_t id_s =
          1u << 4 | 1u << 7 | 1u << 10 | (kTok >> 3) << 17 | (kRow >> 4) << 24;
      // V is MN-major
      constexpr uint32_t id_o =
          1u << 4 | 1u << 7 | 1u << 10 | 1u << 16 | (S::UC * 64 >> 3) << 17 | (kRow >> 4) << 24;
      constexpr int ku = S::DK / S::UC, vu = S::DV / S::UC;  // stages of a K and a V tile
      const uint32_t ring = sb + S::ring;
      Place<S::NST> kp, vp;
      uint32_t tiles = 0;                                // QT 1: tile k has S buffer k % 2
      uint32_t q_ph = 0, p_ph = 0;                       // p_ph: a bit for each S buffer
      const uint32_t q0 = desc_k(sb + S::q);             // [chunk][query tile][128 rows]
      auto landed = [&](const Place<S::NST> &at) {
        wait(bar(S::full) + 8 * at.st, at.ph);
        ptx::fence_proxy_async_smem();
      };
      // S of query tile t into TMEM buffer b against the K tile at kp; Ends: bit 0 the first,
      // bit 1 the last reader of its stages
      auto mma_s = [&](auto t, uint32_t b, auto ends) {
        const uint32_t d = tmem + b * 128;
        Place<S::NST> at = kp;
#pragma unroll
        for (int u = 0; u < ku; ++u) {
          if (ends.v & 1) landed(at);
          if (dead) return;
          const uint32_t k = desc_k(ring + at.st * S::kStage);
#pragma unroll
          for (int x = 0; x < S::UC * 4; ++x)
            ptx::mma_bf16(d,
                          desc(q0 + ((((u * S::UC + (x >> 2)) * S::QT + t.v) * kChunk +
                                      (x & 3) * 32) >> 4)),
                          desc(k + (((x >> 2) * kChunk + (x & 3) * 32) >> 4)), id_s,
                          (u | x) ? 1u : 0u);
          if (ends.v & 2) ptx::mma_commit(bar(S::empty) + 8 * at.st);
          at.advance(1);
        }
        ptx::mma_commit(bar(S::s_full) + 8 * b);
        if (ends.v & 2) kp = at;
      };
      // O of query tile t (+)= P in buffer b times the V tile at vp
      auto mma_o = [&](auto t, uint32_t b, bool first_tile, bool last_tile, auto ends) {
        const uint32_t p = tmem + b * 128, d = tmem + S::o_col + t.v * 128;
        Place<S::NST> at = vp;
        if (ends.v & 1) landed(at);  // before P is, as a rule
        wait(bar(S::p_full) + 16 * b, (p_ph >> b) & 1);
        if (dead) return;
        ptx::tc_fence_after();
#pragma unroll
        for (int u = 0; u < vu; ++u) {
          if ((ends.v & 1) && u > 0) landed(at);
          if (dead) return;
          const uint32_t v = desc_mn(ring + at.st * S::kStage);
#pragma unroll
          for (int x = 0; x < kTok / 16; ++x) {
            if (u == 0 && x == kTok / 32) {
              wait(bar(S::p_full) + 16 * b + 8, (p_ph >> b) & 1);
              if (dead) return;
              ptx::tc_fence_after();
            }
            // P of tokens 0-63 is in columns 32-63 of S, of 64-127 in 96-127
            ptx::mma_bf16_ta(d + u * S::UC * 64, p + 32 + 8 * x + (x < kTok / 32 ? 0 : 32),
                             desc(v + x * (2048 >> 4)), id_o, x ? 1u : (first_tile ? 0u : 1u));
          }
          if (ends.v & 2) ptx::mma_commit(bar(S::empty) + 8 * at.st);
          at.advance(1);
        }
        p_ph ^= 1u << b;
        ptx::mma_commit(bar(S::pv_done + t.v));
        if (last_tile) ptx::mma_commit(bar(S::o_full + t.v));
        if (ends.v & 2) vp = at;
      };
      auto q_done = [&]() {
        if (!dead) ptx::mma_commit(bar(S::q_empty));
      };
      constexpr Int<0> t0;
      constexpr Int<1> t1, first;
      constexpr Int<2> last;
      constexpr Int<3> only;
      while (more) {
        s = after;
        load_q();
        more = walk.next(a, plan, &after);
        const int n = tiles_of(s.tok0, s.tok1, kTokSh);
        // the stages come in the order in which they are read:
        // QT 2: K0 V0 K1 V1 ...; QT 1: K0 K1 V0 K2 V1 ... V(n-1)
        vp = kp;
        vp.advance(S::QT == 1 && n > 1 ? 2 * ku : ku);
        wait(bar(S::q_full), q_ph);
        q_ph ^= 1;
        ptx::fence_proxy_async_smem();
        if (S::QT == 2) {
          if (s.rows > kRow) {
            mma_s(t0, 0, first);
            mma_s(t1, 1, last);
            for (int i = 0; i + 1 < n; ++i) {
              kp.advance(vu);
              mma_o(t0, 0, i == 0, false, first);
              mma_s(t0, 0, first);
              mma_o(t1, 1, i == 0, false, last);
              mma_s(t1, 1, last);
              vp.advance(ku);
            }
            q_done();
            mma_o(t0, 0, n == 1, true, first);
            mma_o(t1, 1, n == 1, true, last);
          } else {
            mma_s(t0, 0, only);
            for (int i = 0; i + 1 < n; ++i) {
              kp.advance(vu);
              mma_o(t0, 0, i == 0, false, only);
              mma_s(t0, 0, only);
              vp.advance(ku);
            }
            q_done();
            mma_o(t0, 0, n == 1, true, only);
          }
        } else {
          mma_s(t0, tiles & 1, only);
          for (int i = 0; i + 1 < n; ++i) {
            if (i > 0) kp.advance(vu);
            mma_s(t0, (tiles + i + 1) & 1, only);
            mma_o(t0, (tiles + i) & 1, i == 0, false, only);
            if (i + 2 < n) vp.advance(ku);
          }
          q_done();
          mma_o(t0, (tiles + n - 1) & 1, n == 1, true, only);
          tiles += n;
        }
        kp = vp;  // the segment's end
      }
      ptx::mma_commit(bar(S::last));  // no MMA is in flight when the TMEM goes back
      if (!ptx::mbar_wait(bar(S::last), 0, kPrefixWaitNs)) *gave_up = 1;
    }
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (*gave_up) {  // copies and MMAs in flight end long before this
    if (tid == 0) {
      atomicOr(a.status, KAMERA_DEVICE_TIMEOUT);
      *a.gave_up = 1;  // the merge writes nothing
    }
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 1000000) {
    }
    __syncthreads();
  }
  if (warp == S::kMma) ptx::tmem_dealloc(tmem, 512);
}

template <class S>
cudaError_t configure() {
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, prefix_tc_kernel<S>);
  if (e != cudaSuccess) return e;
  // the warps' shares come out of the registers that the block is launched with
  if (S::kShift && at.numRegs * S::kThr < S::kRegs) return cudaErrorLaunchOutOfResources;
  return cudaFuncSetAttribute(prefix_tc_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              S::total);
}

template <class S>
cudaError_t launch(const PrefixArgs &a, cudaStream_t s) {
  if (!encode_fn()) return cudaErrorNotSupported;
  Maps m;
  const DevLayout &l = a.lay;
  const int ps = l.page_size, hpk = a.hq / a.n_kv, rb = a.shape.cls[0].rb;
  m.box = ps % kTok == 0 ? kTok : (ps >= 8 && kTok % ps == 0 ? ps : 0);
  const uint32_t box = m.box ? m.box : 8;
  const long long slots = a.pool.num_slots;
  const __nv_bfloat16 *k = a.pool.k + a.layer * slots * l.row_k;
  const __nv_bfloat16 *v = l.kind == KAMERA_GQA ? a.pool.v + a.layer * slots * l.row_v : k;
  const int vrow = l.kind == KAMERA_GQA ? l.row_v : l.row_k;
  bool ok = encode(&m.k, k, 2, l.row_k, slots, 1, l.row_k, 0, box, 1) &&
            encode(&m.v, v, 2, vrow, slots, 1, vrow, 0, box, 1);
  m.q_step = a.n_kv == 1;
  if (m.q_step) {  // a block's rows follow one another
    const uint64_t rows = (uint64_t)a.n_reqs * a.hq;
    const int own = a.hq < rb ? a.hq : rb;
    ok = ok && encode(&m.q_group, a.q, 3, a.dk, 1, rows, a.dk, a.dk, 1, rb) &&
         encode(&m.q_own, a.q, 3, a.dk, 1, rows, a.dk, a.dk, 1, own);
    m.group_bytes = S::DK * 128 * rb;
    m.own_bytes = S::DK * 128 * own;
  } else {
    const uint64_t req = (uint64_t)a.hq * a.dk;
    ok = ok && encode(&m.q_group, a.q, 3, a.dk, a.hq, a.n_reqs, a.dk, req, hpk, rb / hpk) &&
         encode(&m.q_own, a.q, 3, a.dk, a.hq, a.n_reqs, a.dk, req, hpk, 1);
    m.group_bytes = S::DK * 128 * rb;
    m.own_bytes = S::DK * 128 * hpk;
  }
  if (!ok) return cudaErrorInvalidValue;
  return launch_early(prefix_tc_kernel<S>, dim3(a.shape.cls[0].n), S::kThr, S::total, s, a, m);
}

}  // namespace

bool prefix_tc_layout(const DevLayout &l) {
  return (l.kind == KAMERA_GQA && (l.hd == 64 || l.hd == 128)) ||
         (l.kind == KAMERA_MLA && l.latent == 512 && l.rope_d == 64);
}

PrefixClass prefix_tc_class(const DevLayout &l, int hq) {
  const bool gqa = l.kind == KAMERA_GQA;
  const int most = gqa ? 2 * kRow : kRow, hpk = hq / (gqa ? l.H : 1);
  PrefixClass c;
  // several KV heads: whole requests, so that one copy brings a block's queries
  c.rb = gqa && l.H > 1 && hpk > 0 ? most / hpk * hpk : most;
  c.tile_sh = kTokSh;
  c.vh = gqa ? 1 : 2;
  c.n = kSms;
  c.least = 1;
  return c;
}

cudaError_t prepare_prefix_tc(const DevLayout &l) {
  if (l.kind == KAMERA_MLA) return configure<Mla512>();
  return l.hd == 128 ? configure<Gqa128>() : configure<Gqa64>();
}

cudaError_t launch_prefix_tc(const PrefixArgs &a, cudaStream_t s) {
  if (a.lay.kind == KAMERA_MLA) return launch<Mla512>(a, s);
  return a.lay.hd == 128 ? launch<Gqa128>(a, s) : launch<Gqa64>(a, s);
}

}  // namespace kamera
