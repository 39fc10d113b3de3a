// Attention of chunks of new tokens on the tensor cores: GQA with head_dim 64 or 128, MLA with a
// latent of 512 and a rope band of 64. One persistent CTA per SM works its share of tiles off
// (kamera_chunk.cuh); a tile is 128 cached tokens against a block's query rows.
//
//   S [128 rows x 128 tokens] = Q K^T           tcgen05, Q and K from shared memory
//   P = bf16(2^(c S - c m)),  c = |scale| log2 e  a thread to a query row, P into TMEM over S
//   O [128 rows x dims] += P V                   tcgen05, P from TMEM, V from shared memory
//
// The maximum m that P is taken against is raised only when a row's new maximum exceeds it by more
// than 8 / c (a factor of 256 in P, which bf16 and float32 hold without loss); then O is rescaled
// in TMEM. So the weights are taken in one pass over S, against the maximum so far, and only where
// that has to be raised are they taken again. The row sums l take the float32 weights; P is rounded
// to bf16 as the product with V wants it.
//
// Roles: sixteen warps (MLA eight) softmax, rescaling and output, two threads to a query row; one
// (MLA four) brings Q and, through the page table, K and V rows into a ring of stages; a thread for
// each query tile issues the MMAs. Pages of 8, 16, 32 or 64 slots, or a multiple of 128, come as
// tensor-map copies, one per page and 64 columns; pages of V that have tokens no row sees, and other
// page sizes, as 16-byte pieces, zeros where a token has no slot or is not of [first seen, context), so
// that nothing of a row that no token holds is ever multiplied. Tokens that not all rows of a block see
// are: their V times a weight of 0, which is no 0 where V is not finite. Where an output is not finite
// the join kernel therefore looks at V of such tokens, and takes the blocks where one is not finite
// again, token by token (right, and slow: kamera_chunk.cu).
//   GQA: O and S of two query tiles fill the TMEM. A block of more than 128 rows has two tiles of
//        them that share each K and V tile; of a smaller one (requests that decode) the two take
//        turns with the tiles of tokens, each with a maximum, sum and O of its own, joined at the
//        end. Either way the MMAs of one run during the softmax of the other.
//   MLA: one tile of 128 rows and half of V's columns a CTA (O takes 256 TMEM columns; all 512
//        would leave none for S), S of the next tile issued before P V of this one.
// Measured: 2011 new tokens over 60000 (28 query heads, 4 KV heads of 128) at 1280 TFLOP/s, two thirds of
// the dense rate: 3400 cycles a tile of tokens for two query tiles, 2080 of them products, the rest the
// chain from S over the weights to P V that two tiles do not fill (with weights left out 931 us of 1370).
// MLA, 16 heads, 4 x 300 tokens over 9003: 430 us, 5350 cycles a tile for 3330 of products: Q leaves
// room for five stages of 16 KB, and a tile takes thirteen. With a thread and a ring of its own for K
// (three stages) and for V (two) 457 us: the ring's latency counts, not the issue.
// Layout: every operand tile is 128 rows of 128 bytes (64 elements), swizzled in 128-byte rows;
// V is read MN-major, so its rows land unchanged too.
#include "kamera_chunk.cuh"
#include "kamera_ptx.cuh"
#include "kamera_smem.cuh"
#include "kamera_tc.cuh"

namespace kamera {

namespace {

constexpr int kTokSh = 7, kTok = 1 << kTokSh;  // tokens per tile
constexpr int kRow = 128;              // query rows per MMA
constexpr int kMasks = 8;              // tiles whose token masks are kept
constexpr int kSegs = 8;               // segments that are kept

// DK, DV: 64-column chunks of K and of the CTA's V columns; QT: tiles of query rows; UC: chunks
// per ring stage; NST: ring stages; NL: warps that load K and V.
template <int DK_, int DV_, int QT_, int UC_, int NST_, int NL_>
struct Shape {
  static constexpr int DK = DK_, DV = DV_, QT = QT_, UC = UC_, NST = NST_, NL = NL_;
  // softmax warps; NL loading warps, an MMA warp for each query tile
  static constexpr int kSoft = 8 * QT, kMma = kSoft + NL;
  static constexpr bool kTwo = QT == 2;
  static constexpr int kThr = 32 * (kTwo ? (kMma + QT + 3) / 4 * 4 : kMma + QT);
  // With two query tiles the softmax warps take registers of the others; whole warpgroups
  static constexpr int kRegsSoft = 104, kRegsRest = 64;
  static constexpr int kRegs = 32 * kSoft * kRegsSoft + (kThr - 32 * kSoft) * kRegsRest;
  static constexpr int kStage = UC * kChunk;
  static constexpr int q = 0;
  static constexpr int ring = QT * DK * kChunk;
  static constexpr int mask = ring + NST * kStage;  // uint32 [kMasks][4]
  static constexpr int xch = mask + kMasks * 16;    // float [2 QT][kRow]: maxima, sums
  static constexpr int bar = xch + 2 * QT * kRow * 4;
  // mbarriers
  static constexpr int full = 0, empty = NST, q_full = empty + NST, q_empty = q_full + 1,
                       s_full = q_empty + 1, p_full = s_full + 2, pv_done = p_full + 2,
                       o_free = pv_done + 1, o_full = o_free + 1,
                       mk_full = o_full + 2, sg_full = mk_full + kMasks, last = sg_full + kSegs,
                       turn = last + 2, n_bar = turn + 2;
  static constexpr int misc = bar + n_bar * 8;  // TMEM address, give-up flag, odd values
  static constexpr int walk = misc + 16;        // ChunkWalk
  static constexpr int seg = walk + sizeof(ChunkWalk);  // ChunkSegment [kSegs]
  static constexpr int total = seg + kSegs * sizeof(ChunkSegment);
  static constexpr int scratch = xch;           // of the start
  static constexpr uint32_t o_col = 256;        // O of tile t at o_col + t * 128
  static_assert(total <= 232448, "shared memory of one CTA");
  static_assert(DK % UC == 0 && DV % UC == 0, "whole stages");
  static_assert(scratch % 8 == 0 && walk % 8 == 0, "of 64-bit numbers");
  static_assert(sizeof(ChunkScratch<kThr>) <= bar - xch, "the start's scratch");
  static_assert(!kTwo || kThr % 128 == 0, "whole warpgroups");
};

using Gqa128 = Shape<2, 2, 2, 2, 5, 1>;
using Gqa64 = Shape<1, 1, 2, 1, 10, 1>;
using Mla512 = Shape<9, 4, 1, 1, 5, 4>;

// Tensor maps of a call: pool rows of the layer (boxes of 64 columns and `box` slots) and query
// rows (64 columns of a block's heads, of all its tokens or of one).
struct Maps {
  CUtensorMap k, v, q_block, q_token;
  int box;                       // slots per copy; 0: rows come by cp.async
  int copies, per_page;          // of a tile's 64 columns; tiles of a page, where that is one
  int block_bytes, token_bytes;  // of the query copies
};

template <class S>
__global__ void __launch_bounds__(S::kThr, 1) chunk_tc_kernel(
    const __grid_constant__ ChunkArgs a, const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = ptx::smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const DevLayout &lay = a.lay;
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + S::misc);
  volatile uint32_t *gave_up = misc + 1;
  volatile uint32_t *odd = misc + 2;
  const ChunkPlaces places = chunk_places(a.shape, a.ws);
  auto bar = [&](int i) { return sb + S::bar + 8 * i; };
  // Waits for a phase, giving up after a.wait_ns or when another thread has. A thread that gave up
  // runs on to the end of its segment without waiting, arriving, copying or multiplying: it keeps step
  // with the named barriers only, and no barrier gets an arrival that it does not expect. Threads that
  // meet (a warp, the softmax warps) leave together.
  bool dead = false;
  auto wait = [&](uint32_t b, uint32_t parity) {
    if (__builtin_expect(dead || ptx::mbar_try_wait(b, parity), 1)) return;
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait_for(b, parity, 20000)) {
      if (*gave_up || ptx::globaltimer() - t0 > a.wait_ns) {
        *gave_up = 1;
        dead = true;
        return;
      }
    }
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
      ptx::mbar_init(bar(S::full + i), 32);
      ptx::mbar_init(bar(S::empty + i), S::QT);
    }
    ptx::mbar_init(bar(S::q_full), 1);
    ptx::mbar_init(bar(S::q_empty), S::QT);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(S::s_full + i), 1);
      ptx::mbar_init(bar(S::p_full + i), 8);
      ptx::mbar_init(bar(S::o_full + i), 1);
    }
    ptx::mbar_init(bar(S::pv_done), 1);
    ptx::mbar_init(bar(S::o_free), S::kSoft);
    for (int i = 0; i < kMasks; ++i) ptx::mbar_init(bar(S::mk_full + i), 1);
    for (int i = 0; i < kSegs; ++i) ptx::mbar_init(bar(S::sg_full + i), 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(bar(S::last + i), 1);
      ptx::mbar_init(bar(S::turn + i), 1);
    }
    ptx::fence_mbar_init();
    ptx::mbar_arrive(bar(S::turn));  // the first query tile begins
    *gave_up = !begins;
    *odd = 0;
    ptx::prefetch_map(&maps.k);
    ptx::prefetch_map(&maps.v);
    ptx::prefetch_map(&maps.q_block);
    ptx::prefetch_map(&maps.q_token);
  }
  const ChunkStart st = chunk_start<S::kThr>(
      a, blockIdx.x, reinterpret_cast<ChunkScratch<S::kThr> *>(smem + S::scratch));
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];
  ptx::launch_dependents();
  // The worker's segments. The loading warp walks them (in shared memory, as a walk would take
  // registers of all) and publishes each after the first tile of the one before; a segment
  // with no tiles ends them. With kSegs places the one that is overwritten has been left by all: a
  // segment takes two stages or more, and its last V stage is free only after O of the segment
  // before has been read.
  ChunkWalk *walk = reinterpret_cast<ChunkWalk *>(smem + S::walk);
  ChunkSegment *segs = reinterpret_cast<ChunkSegment *>(smem + S::seg);
  uint32_t seg_no = 0;  // segments taken
  auto take_segment = [&]() -> const ChunkSegment * {  // the next one, null behind the last
    const uint32_t k = seg_no % kSegs;
    wait(bar(S::sg_full + k), seg_no / kSegs & 1);
    const ChunkSegment *s = segs + k;
    if (dead || s->t0 == s->t1) return nullptr;
    ++seg_no;
    return s;
  };
  // The same for a whole warp: of its threads one alone may have given up (the elected one, on a stage),
  // and none may leave while the others go on to what they do together.
  auto take_whole = [&]() -> const ChunkSegment * {
    const ChunkSegment *s = take_segment();
    dead = __any_sync(0xffffffffu, dead);
    return dead ? nullptr : s;
  };
  // And for all softmax warps, which meet at named barriers in every segment. What they have read of the
  // exchange buffer in the segment before, too, they have read before any of them writes to it again.
  // (Three prompts of 4001 tokens, 8 blocks a CTA: 328 us without this barrier, 333 with it.)
  auto take_together = [&]() -> const ChunkSegment * {
    const ChunkSegment *s = take_segment();
    return ptx::barrier_or(2, 32 * S::kSoft, dead) ? nullptr : s;
  };
  if (warp == S::kSoft) {
    ChunkWalk w;
    w.start(a, st, blockIdx.x);
    if (!begins) w.left = 0;
    if (lane == 0) *walk = w;
    __syncwarp();
  }

  if (warp < S::kSoft) {
    if (S::kTwo) ptx::regs_more<S::kRegsSoft>();
    // ---- softmax: two threads (of two warps) to a query row, kCols tokens of each tile and half of
    // O's columns each; of two query tiles each has warps of its own ----
    constexpr int kCols = kTok / 2, kOut = S::DV * 32;
    const int w = warp >> 3;                       // query tile
    const int qr = (warp >> 2) & 1;                // the thread's half of the tokens and columns
    const int lane_row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    // (a scale of 0 is one that makes nothing of any score: -inf, where a token is not seen, times
    // it is -inf)
    const float c = fmaxf(fabsf(a.scale) * kLog2e, 1.2e-38f);
    const bool flip = a.scale < 0.f;
    const float inf = __int_as_float(0x7f800000);
    float *xch = reinterpret_cast<float *>(smem + S::xch) + 2 * w * kRow;  // [half][row]
    const int pair = 3 + w * 4 + (warp & 3);  // named barrier of a row's two warps
    auto arrive = [&](uint32_t b) {  // once for the warp
      __syncwarp();
      if (lane == 0 && !dead) ptx::mbar_arrive(b);
    };
    uint32_t mine = 0;   // tiles of this warp so far: phases of its buffers
    uint32_t seen = 0;   // tiles of the CTA's segments so far
    ChunkSegment last = {};
    while (const ChunkSegment *sp = take_together()) {
      const ChunkSegment &s = *sp;
      const uint32_t parity = (seg_no - 1) & 1;
      if (tid == 0) last = s;
      const int n = s.t1 - s.t0, tile0 = s.t0, rows = s.ntok * s.heads;
      const bool turns = S::kTwo && rows <= kRow;  // the tiles of tokens in turn
      const int i_row = (turns ? 0 : kRow * w) + lane_row;
      const bool live = i_row - lane < rows;  // a warp without rows only keeps step
      int tok, h;
      chunk_row(a, s, i_row < rows ? i_row : 0, &tok, &h);
      // a thread without a row sees all, against a maximum that leaves nothing
      const int see1 = i_row < rows ? s.first + tok + 1 : 0x7FFFFFFF;
      const int see0 = i_row < rows ? first_seen(a, s.first + tok) : 0;
      // tiles of which all the warp's rows see the warp's half
      const int in0 = (__reduce_max_sync(0xffffffffu, see0) - kCols * qr + kTok - 1) >> kTokSh;
      const int in1 =
          flip ? 0 : (__reduce_min_sync(0xffffffffu, see1) - kCols * (qr + 1) + kTok) >> kTokSh;
      float m = i_row < rows ? -inf : inf;
      f32x2 la = f2(0.f, 0.f), lb = la;
      const uint32_t o_t = tmem + S::o_col + w * 128 + lane_off + qr * kOut;
      bool done = false;  // a tile of this segment
      for (int i = turns ? w : 0; i < n; i += turns ? 2 : 1, ++mine) {
        const uint32_t b = S::kTwo ? w : mine & 1;
        uint2 msk;
        bool plain;
        // The tile's mask. It is there before S is; of a segment's first tile it is read after S, as
        // this thread may be more tiles ahead of the loader than masks are kept
        auto read_mask = [&]() {
          const uint32_t mk = (seen + i) % kMasks;
          wait(bar(S::mk_full) + 8 * mk, (seen + i) / kMasks & 1);
          __syncwarp();
          msk = *reinterpret_cast<const uint2 *>(smem + S::mask + 16 * mk + 8 * qr);
          plain = tile0 + i >= in0 && tile0 + i < in1 && (msk.x & msk.y) == 0xffffffffu;
        };
        if (live && done) read_mask();
        wait(bar(S::s_full) + 8 * b, (S::kTwo ? mine : mine >> 1) & 1);
        __syncwarp();
        ptx::tc_fence_after();
        if (live) {
          const uint32_t s_t = tmem + b * 128 + qr * kCols + lane_off;
          uint32_t x[32];
          ptx::tmem_ld32(s_t, x);
          if (!done) read_mask();
          if (__builtin_expect(!plain, 0)) {
            const int t0 = ((tile0 + i) << kTokSh) + kCols * qr;
            auto seen_of = [&](int from, int to) {  // of 32 tokens, those in [from, to)
              const uint32_t up = from <= 0 ? 0xffffffffu : from >= 32 ? 0u : 0xffffffffu << from;
              const uint32_t dn = to >= 32 ? 0xffffffffu : to <= 0 ? 0u : (1u << to) - 1u;
              return up & dn;
            };
            msk.x &= seen_of(see0 - t0, see1 - t0);
            msk.y &= seen_of(see0 - t0 - 32, see1 - t0 - 32);
          }
          float base = m > -inf ? m * c : 0.f;
          uint32_t p[kCols / 2];
          f32x2 ha, hb;       // this tile's sums
          float top;
          // The weights against `base`, their sums and the maximum on the way, 32 columns of S at a
          // time, the first already on their way into x
          auto weights = [&]() {
            ha = hb = f2(0.f, 0.f);
            float t0 = -inf, t1 = -inf;
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              if (g) ptx::tmem_ld32(s_t + 32, x);
              ptx::tmem_ld_wait_all<32>(x);
              if (__builtin_expect(!plain, 0)) {
                if (flip) {
#pragma unroll
                  for (int e = 0; e < 32; ++e) x[e] ^= 0x80000000u;
                }
                const uint32_t bits = g ? msk.y : msk.x;
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = bits & (1u << e) ? x[e] : 0xff800000u;
              }
#pragma unroll
              for (int e = 0; e < 32; e += 2) {
                const float y0 = __uint_as_float(x[e]), y1 = __uint_as_float(x[e + 1]);
                const float p0 = exp2_approx(fmaf(y0, c, -base));
                const float p1 = exp2_approx(fmaf(y1, c, -base));
                float &t = e & 2 ? t1 : t0;
                t = fmaxf(fmaxf(t, y0), y1);
                if (e & 2)
                  hb = add2(hb, f2(p0, p1));
                else
                  ha = add2(ha, f2(p0, p1));
                p[16 * g + e / 2] = pack_bf16(p0, p1);
              }
            }
            top = fmaxf(t0, t1);
          };
          weights();
          // the weights stand unless the maximum is to be raised, for either half of the row
          if (__builtin_expect(
                  ptx::barrier_or(pair, 64, (m == -inf && top > -inf) || (top - m) * c > 8.f), 0)) {
            xch[qr * kRow + lane_row] = top;
            ptx::barrier_sync(pair, 64);
            top = fmaxf(top, xch[(qr ^ 1) * kRow + lane_row]);
            const bool first = m == -inf && top > -inf;
            const bool up = first || (top - m) * c > 8.f;
            const float f = up ? (first ? 0.f : exp2_approx((m - top) * c)) : 1.f;
            if (up) m = top;
            la = fma2(la, f2(f, f), f2(0.f, 0.f));
            lb = fma2(lb, f2(f, f), f2(0.f, 0.f));
            if (done) {
              // P V of the tile before is complete: S of this one says so, where it was issued
              // behind it (else S says so of the one before that, and the parity is unambiguous)
              if (!S::kTwo) {
                wait(bar(S::pv_done), (mine - 1) & 1);
                __syncwarp();
                ptx::tc_fence_after();
              }
#pragma unroll 1
              for (int j = 0; j < kOut; j += 16) {
                uint32_t z[16];
                ptx::tmem_ld16(o_t + j, z);
                ptx::tmem_ld_wait_all<16>(z);
#pragma unroll
                for (int e = 0; e < 16; ++e) z[e] = __float_as_uint(__uint_as_float(z[e]) * f);
                ptx::tmem_st16(o_t + j, z);
              }
              ptx::tmem_st_wait();
            }
            // (what a row's threads have scaled is multiplied after both have arrived)
            ptx::barrier_sync(pair, 64);
            base = m > -inf ? m * c : 0.f;
            ptx::tmem_ld32(s_t, x);
            weights();
          }
          la = add2(la, ha);
          lb = add2(lb, hb);
          ptx::tmem_st32(s_t, p);  // P over its half of S
          ptx::tmem_st_wait();
        }
        ptx::tc_fence_before();
        arrive(bar(S::p_full) + 8 * b);
        done = true;
      }
      seen += n;
      // ---- output ----
      wait(bar(S::o_full) + 8 * w, parity);
      if (turns) wait(bar(S::o_full) + 8 * (w ^ 1), parity);
      __syncwarp();
      ptx::tc_fence_after();
      float l, f0 = 1.f, f1 = 0.f;  // factors of this query tile's O and of the other's
      {
        float l0, l1;
        f2_split(add2(la, lb), l0, l1);
        l = l0 + l1;
      }
      if (turns) {  // the two turns' sums and O are joined
        float *all = reinterpret_cast<float *>(smem + S::xch) + lane_row;
        xch[qr * kRow + lane_row] = m;
        ptx::barrier_sync(2, 4 * kRow);
        const float mo = all[2 * (w ^ 1) * kRow], top = fmaxf(m, mo);  // (never NaN)
        f0 = m == -inf ? 0.f : exp2_approx((m - top) * c);
        f1 = mo == -inf ? 0.f : exp2_approx((mo - top) * c);
        m = top;
        ptx::barrier_sync(2, 4 * kRow);
        xch[qr * kRow + lane_row] = n > w ? l * f0 : 0.f;
        ptx::barrier_sync(2, 4 * kRow);
        l = (all[0] + all[kRow]) + (all[2 * kRow] + all[3 * kRow]);
      } else if (live) {
        xch[qr * kRow + lane_row] = l;
        ptx::barrier_sync(pair, 64);
        l = xch[lane_row] + xch[kRow + lane_row];
      }
      if (live) {
        const bool ok = l != 0.f && !*gave_up;
        const float inv = 1.f / l, g0 = f0 * inv, g1 = f1 * inv;
        const bool whole = chunk_whole(s), whole32 = (reinterpret_cast<uintptr_t>(a.out) & 31) == 0;
        const long long rh = (long long)(s.row + tok) * a.hq + h;
        const long long place = (long long)(2 * blockIdx.x + (s.carry() ? 0 : 1)) * a.shape.rb + i_row;
        __nv_bfloat16 *out = a.out + rh * a.dv + s.part * a.shape.vw;
        float *part = places.o + place * a.shape.vw;
        const bool write = i_row < rows && !*gave_up;
        // of a row's columns, this thread's: half, in turns a quarter
        const int cols = kOut / (turns ? 2 : 1), from = (turns ? 2 * w + qr : qr) * cols;
        const bool has = !turns || n > w, other = turns && n > 1 - w;
        const uint32_t o_mine = tmem + S::o_col + lane_off + w * 128;
        const uint32_t o_other = tmem + S::o_col + lane_off + (w ^ 1) * 128;
        float odd_sum = 0.f;
#pragma unroll 1
        for (int j = from; j < from + cols; j += 16) {
          uint32_t z[16];
          ptx::tmem_ld16(o_mine + j, z);
          ptx::tmem_ld_wait_all<16>(z);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            z[e] = ok && has ? __float_as_uint(__uint_as_float(z[e]) * g0) : 0u;
          if (other) {
            uint32_t z1[16];
            ptx::tmem_ld16(o_other + j, z1);
            ptx::tmem_ld_wait_all<16>(z1);
#pragma unroll
            for (int e = 0; e < 16; ++e)
              z[e] = ok ? __float_as_uint(fmaf(__uint_as_float(z1[e]), g1, __uint_as_float(z[e])))
                        : 0u;
          }
#pragma unroll
          for (int e = 0; e < 16; ++e) odd_sum = fmaf(__uint_as_float(z[e]), 0.f, odd_sum);
          if (write && whole) {
            uint32_t u[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              u[e] = pack_bf16(__uint_as_float(z[2 * e]), __uint_as_float(z[2 * e + 1]));
            if (whole32) {
              ptx::stg32(out + j, u);
            } else {
              *reinterpret_cast<uint4 *>(out + j) = make_uint4(u[0], u[1], u[2], u[3]);
              *reinterpret_cast<uint4 *>(out + j + 8) = make_uint4(u[4], u[5], u[6], u[7]);
            }
          } else if (write) {
            ptx::stg32(part + j, z);
            ptx::stg32(part + j + 8, z + 8);
          }
        }
        if (write && odd_sum != 0.f) *odd = 1;
        if (write && from == 0) {
          const float z = l != 0.f ? (m * c + log2f(l)) * kLn2 : -inf;
          if (!whole)
            places.lse[place] = z;
          else if (s.part == 0)
            a.lse[rh] = z;
        }
      }
      ptx::tc_fence_before();
      arrive(bar(S::o_free));
    }
    if (tid == 0)
      chunk_note(places.rec + blockIdx.x, last, seg_no, false, false);
  } else if (warp < S::kMma) {
    if (S::kTwo) ptx::regs_fewer<S::kRegsRest>();
    // ---- Q, and K and V rows into the ring: a warp issues the sixteen copies of a 32 KB stage in
    // about 450 cycles. What a warp does alone takes about five cycles an instruction, so whole tiles
    // take as few as may be: a lane to a page, one load and one test ahead of its tile. Copies are
    // issued by one thread, which stands in for the others' arrivals. Several warps (MLA) bring a stage
    // in turn ----
    const int part = warp - S::kSoft;
    const bool gqa = lay.kind == KAMERA_GQA;
    const int box = maps.box, each = maps.copies;  // slots of a copy, copies of a tile's 64 columns
    const int per_page = maps.per_page;            // tiles of a page (each == 1)
    const unsigned pages = (unsigned)(a.pool.num_slots / lay.page_size);
    const uint32_t all_pages = box ? (1u << each) - 1u : 0xffffffffu;
    Place<S::NST> at;            // the next stage
    uint32_t stage_no = 0;       // of that stage, since the start: every NL-th is a warp's
    uint32_t tile_no = 0;        // tiles so far
    uint32_t published = 0;
    auto publish = [&]() {       // the next segment
      if (part == 0 && lane == 0) {
        ChunkSegment *to = segs + published % kSegs;
        if (!walk->next(a, to)) to->t0 = to->t1 = 0;
        if (!dead) ptx::mbar_arrive(bar(S::sg_full) + 8 * (published % kSegs));
      }
      ++published;
      __syncwarp();
    };
    publish();
    while (const ChunkSegment *sp = take_whole()) {
      const int n = sp->t1 - sp->t0, tile0 = sp->t0, ctx = sp->ctx;
      const int kcol = gqa ? sp->kvh * lay.hd : 0, vcol = kcol + sp->part * a.shape.vw;
      const int lo = first_seen(a, sp->first);  // tokens that a row sees: from here on
      const int *table = a.pool.pt + (long long)sp->r * a.pool.pt_stride;
      // the lane's page-table entry in a tile, -1 where none of the page's tokens is in [lo, ctx)
      auto load_entry = [&](int i) {
        const long long tok = ((long long)(tile0 + i) << kTokSh) + lane * box;
        const bool on = i < n && lane < each && tok + box > lo && tok < ctx;
        const int t = tile0 + i;
        return on ? __ldg(table + (each == 1 ? t / per_page : t * each + lane)) : -1;
      };
      int entry = box ? load_entry(0) : -1;
      struct Tile {
        int y;           // first slot of the lane's page
        uint32_t pages;  // pages of the pool with tokens in [lo, ctx), a bit each
        uint32_t inner;  // those with no others
      } cur, prev;
      cur.y = 0;
      cur.pages = cur.inner = 0;
      // slots of four tokens of a tile, for those that come piece by piece
      auto slots = [&](int i, int *to) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const long long tok = ((long long)(tile0 + i) << kTokSh) + 32 * k + lane;
          to[k] = tok >= lo && tok < ctx ? slot_in(a, load_page(a, sp->r, (int)tok), (int)tok) : -1;
        }
      };
      auto bring = [&](bool is_k, int i, const Tile &tile) {
        const int col = is_k ? kcol : vcol, stages = (is_k ? S::DK : S::DV) / S::UC;
        const void *map = is_k ? &maps.k : &maps.v;
        // What is in K's rows that no token of [lo, ctx) has does not matter, as a token's scores are
        // a column of their own and such columns are masked. V's have to be 0: a weight of 0 times
        // what is not finite is no 0.
        const uint32_t copied = is_k ? tile.pages : tile.pages & tile.inner;
        if (copied == all_pages) {
          int y[16];
#pragma unroll
          for (int k = 0; k < 16; ++k) y[k] = __shfl_sync(0xffffffffu, tile.y, k);
          if (ptx::elect_one()) {
            Place<S::NST> to = at;
#pragma unroll 1
            for (int u = 0; u < stages; ++u, to.advance(1)) {
              if (S::NL > 1 && (stage_no + u) % S::NL != part) continue;  // another warp's
              const uint32_t full = bar(S::full) + 8 * to.st;
              uint32_t dst = sb + S::ring + to.st * S::kStage;
              wait(bar(S::empty) + 8 * to.st, to.ph ^ 1);
              if (dead) break;
              ptx::mbar_arrive_n(full, 31);
              ptx::mbar_arrive_expect_tx(full, S::kStage);
#pragma unroll
              for (int k = 0; k < 16; ++k) {
                if (k >= each) break;
#pragma unroll
                for (int c = 0; c < S::UC; ++c)
                  ptx::tma_2d(dst + c * kChunk, map, col + (u * S::UC + c) * 64, y[k], full);
                dst += box * 128;
              }
            }
          }
          __syncwarp();
          at.advance(stages);
          stage_no += stages;
          return;
        }
        const __nv_bfloat16 *base = is_k || !gqa ? a.pool.k : a.pool.v;
        const int row = is_k || !gqa ? lay.row_k : lay.row_v;
        const int piece = lane & 7;  // 16-byte piece of a row
        base += (long long)a.layer * a.pool.num_slots * row + col + 8 * piece;
        if (box) {
          const long long t0 = (long long)(tile0 + i) << kTokSh;
#pragma unroll 1
          for (int u = 0; u < stages; ++u, at.advance(1), ++stage_no) {
            if (S::NL > 1 && stage_no % S::NL != part) continue;
            const uint32_t full = bar(S::full) + 8 * at.st;
            const uint32_t dst = S::ring + at.st * S::kStage;
            wait(bar(S::empty) + 8 * at.st, at.ph ^ 1);
            if (__any_sync(0xffffffffu, dead)) {
              dead = true;
              continue;
            }
            if (lane == 0) ptx::mbar_arrive_expect_tx(full, __popc(copied) * box * S::UC * 128);
            __syncwarp();
#pragma unroll 1
            for (int k = 0; k < each; ++k) {
              const int first = __shfl_sync(0xffffffffu, tile.y, k);
              if (copied >> k & 1) {
                if (ptx::elect_one())
#pragma unroll
                  for (int c = 0; c < S::UC; ++c)
                    ptx::tma_2d(sb + dst + c * kChunk + k * box * 128, map,
                                col + (u * S::UC + c) * 64, first, full);
                __syncwarp();
              } else if (!is_k) {
#pragma unroll 4
                for (int j = lane >> 3; j < box; j += 4) {  // four tokens at a time
                  const int t = k * box + j;
                  const bool has = tile.pages >> k & 1 && t0 + t >= lo && t0 + t < ctx;
#pragma unroll
                  for (int c = 0; c < S::UC; ++c) {
                    uint4 v = make_uint4(0, 0, 0, 0);
                    if (has)
                      v = __ldg(reinterpret_cast<const uint4 *>(
                          base + (long long)(first + j) * row + (u * S::UC + c) * 64));
                    *reinterpret_cast<uint4 *>(smem + dst + c * kChunk + t * 128 +
                                               ((piece ^ (t & 7)) << 4)) = v;
                  }
                }
                __syncwarp();
              }
            }
            ptx::fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive_n(full, 31);
          }
          return;
        }
        int slot[4];
        slots(i, slot);
#pragma unroll 1
        for (int u = 0; u < stages; ++u, at.advance(1), ++stage_no) {
          if (S::NL > 1 && stage_no % S::NL != part) continue;
          const uint32_t dst = sb + S::ring + at.st * S::kStage, full = bar(S::full) + 8 * at.st;
          wait(bar(S::empty) + 8 * at.st, at.ph ^ 1);
          if (__any_sync(0xffffffffu, dead)) {
            dead = true;
            continue;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll 2
            for (int j = 0; j < 8; ++j) {  // four tokens at a time
              const int t = 32 * k + 4 * j + (lane >> 3);
              const int sl = __shfl_sync(0xffffffffu, slot[k], 4 * j + (lane >> 3));
              const __nv_bfloat16 *p = base + (long long)max(sl, 0) * row + u * S::UC * 64;
#pragma unroll
              for (int c = 0; c < S::UC; ++c)
                ptx::cp_async16(dst + c * kChunk + t * 128 + ((piece ^ (t & 7)) << 4), p + c * 64,
                                sl >= 0 ? 16u : 0u);
            }
          // made visible to the tensor core here, as the MMA thread does not stop for it
          ptx::cp_async_commit();
          ptx::cp_async_wait_all();
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(full);
        }
      };
      if (part == 0) {
        // Q, once S of the segment before is complete. Rows of a copy past the block's are other
        // tokens' or zero: their results go nowhere
        if (seg_no > 1) wait(bar(S::q_empty), seg_no & 1);
        if (!__any_sync(0xffffffffu, dead) && ptx::elect_one()) {
          const bool one = sp->ntok == 1;
          ptx::mbar_arrive_expect_tx(bar(S::q_full), one ? maps.token_bytes : maps.block_bytes);
          for (int c = 0; c < S::DK; ++c)
            ptx::tma_3d(sb + S::q + c * S::QT * kChunk, one ? &maps.q_token : &maps.q_block,
                        c * 64, sp->h0, sp->row, bar(S::q_full));
        }
        __syncwarp();
      }
      // the stages come in the order K0 V0 K1 V1 ..., in MLA's one query tile, whose tiles take more
      // stages than there are, in that in which they are read: K0 K1 V0 K2 V1 ... V(n-1)
#pragma unroll 1
      for (int i = 0; i < n; ++i) {
        const uint32_t mk = tile_no++ % kMasks;
        const long long t0 = (long long)(tile0 + i) << kTokSh;
        prev = cur;
        uint4 bits;
        if (box) {
          const long long tok = t0 + lane * box;
          const bool on = lane < each && tok + box > lo && tok < ctx, in = (unsigned)entry < pages;
          if (on && !in) atomicOr(a.status, KAMERA_DEVICE_SLOT_OOB);
          cur.y = entry * lay.page_size + (each == 1 ? (tile0 + i) % per_page * kTok : 0);
          cur.pages = __ballot_sync(0xffffffffu, on && in);
          cur.inner = __ballot_sync(0xffffffffu, on && tok >= lo && tok + box <= ctx);
          if (i + 1 < n) entry = load_entry(i + 1);  // ahead of its use
          if ((cur.pages & cur.inner) == all_pages) {
            bits = make_uint4(0xffffffffu, 0xffffffffu, 0xffffffffu, 0xffffffffu);
          } else {
            auto word = [&](int k) {  // of 32 tokens, those that are in
              const int t = 32 * k + lane;
              return __ballot_sync(0xffffffffu, (cur.pages >> (t / box) & 1) && t0 + t >= lo &&
                                                    t0 + t < ctx);
            };
            bits = make_uint4(word(0), word(1), word(2), word(3));
          }
        } else {
          int slot[4];
          slots(i, slot);
          bits.x = __ballot_sync(0xffffffffu, slot[0] >= 0);
          bits.y = __ballot_sync(0xffffffffu, slot[1] >= 0);
          bits.z = __ballot_sync(0xffffffffu, slot[2] >= 0);
          bits.w = __ballot_sync(0xffffffffu, slot[3] >= 0);
        }
        if (part == 0 && lane == 0) {
          *reinterpret_cast<uint4 *>(smem + S::mask + 16 * mk) = bits;
          if (!dead) ptx::mbar_arrive(bar(S::mk_full) + 8 * mk);
        }
        __syncwarp();
        bring(true, i, cur);
        if (i == 0) publish();
        if (S::kTwo)
          bring(false, i, cur);
        else if (i > 0)
          bring(false, i - 1, prev);
      }
      if (!S::kTwo) bring(false, n - 1, cur);
    }
    ptx::cp_async_wait_all();
  } else {
    if (S::kTwo) ptx::regs_fewer<S::kRegsRest>();
    // ---- MMAs, one thread for each query tile: a wait, a commit and the way round the loop take it
    // some hundred cycles each, and while it is on them the other's products go on. The descriptors of
    // a tile's steps differ by constants ----
    if (warp < S::kMma + S::QT && ptx::elect_one()) {
      const int t = warp - S::kMma;
      constexpr uint32_t id_s =
          1u << 4 | 1u << 7 | 1u << 10 | (kTok >> 3) << 17 | (kRow >> 4) << 24;
      // V is MN-major
      constexpr uint32_t id_o =
          1u << 4 | 1u << 7 | 1u << 10 | 1u << 16 | (S::UC * 64 >> 3) << 17 | (kRow >> 4) << 24;
      constexpr int ku = S::DK / S::UC, vu = S::DV / S::UC;  // stages of a K and a V tile
      const uint32_t ring = sb + S::ring;
      Place<S::NST> kp;                                  // the next K tile (two query tiles: stage)
      uint32_t tiles = 0;                                // tiles so far; one query tile: k has S buffer
                                                         // k % 2
      uint32_t p_ph = 0;                                 // a bit for each S buffer
      auto commit = [&](int b) {
        if (!dead) ptx::mma_commit(bar(b));
      };
      // S of the query tile at qt into TMEM buffer b against the K tile at `at`; `passes` is called
      // when the MMAs have been issued
      auto mma_s = [&](uint32_t qt, uint32_t b, Place<S::NST> &at, auto passes) {
        const uint32_t d = tmem + b * 128;
#pragma unroll
        for (int u = 0; u < ku; ++u) {
          wait(bar(S::full) + 8 * at.st, at.ph);
          if (dead) return;
          const uint32_t k = desc_k(ring + at.st * S::kStage);
#pragma unroll
          for (int x = 0; x < S::UC * 4; ++x)
            ptx::mma_bf16(
                d, desc(qt + (((u * S::UC + (x >> 2)) * S::QT * kChunk + (x & 3) * 32) >> 4)),
                desc(k + (((x >> 2) * kChunk + (x & 3) * 32) >> 4)), id_s, (u | x) ? 1u : 0u);
          if (u == ku - 1) {
            passes();
            ptx::mma_commit(bar(S::s_full) + 8 * b);
          }
          ptx::mma_commit(bar(S::empty) + 8 * at.st);
          at.advance(1);
        }
      };
      // What O of that buffer waits for.
      auto ready_o = [&](uint32_t b, const Place<S::NST> &at) {
        wait(bar(S::full) + 8 * at.st, at.ph);  // before P is, as a rule
        wait(bar(S::p_full) + 8 * b, p_ph >> b & 1);
        p_ph ^= 1u << b;
      };
      // O at d (+)= P in buffer b times the V tile at `at`
      auto mma_o = [&](uint32_t d, uint32_t b, bool first_tile, Place<S::NST> &at) {
        const uint32_t p = tmem + b * 128;
        if (dead) return;
        ptx::tc_fence_after();
#pragma unroll
        for (int u = 0; u < vu; ++u) {
          if (u > 0) wait(bar(S::full) + 8 * at.st, at.ph);
          if (dead) return;
          const uint32_t v = desc_mn(ring + at.st * S::kStage);
#pragma unroll
          for (int x = 0; x < kTok / 16; ++x) {
            // P of tokens 0-63 is in columns 0-31 of S, of 64-127 in 64-95
            ptx::mma_bf16_ta(d + u * S::UC * 64, p + 8 * x + (x < kTok / 32 ? 0 : 32),
                             desc(v + x * (2048 >> 4)), id_o, x ? 1u : (first_tile ? 0u : 1u));
          }
          ptx::mma_commit(bar(S::empty) + 8 * at.st);
          at.advance(1);
        }
        if (!S::kTwo) ptx::mma_commit(bar(S::pv_done));
      };
      uint32_t turns = 0;  // of this thread so far
      auto pass = [&]() {
        if (!dead) ptx::mbar_arrive(bar(S::turn) + 8 * (t ^ 1));
      };
      auto stay = []() {};
      const uint32_t q0 = desc_k(sb + S::q);  // [chunk][query tile][128 rows]
      while (const ChunkSegment *sp = take_segment()) {
        const int n = sp->t1 - sp->t0;
        const bool before = seg_no > 1;
        auto o_free = [&]() {  // O of the segment before has been read
          if (before) wait(bar(S::o_free), seg_no & 1);
        };
        wait(bar(S::q_full), (seg_no - 1) & 1);
        if constexpr (S::kTwo) {
          const bool pairs = sp->ntok * sp->heads > kRow;
          const uint32_t o = tmem + S::o_col + t * 128;
          if (pairs) {
            // Of a pair of query tiles each takes every tile of tokens. They go in turn, each P V of
            // its tile before and S of the next: without an order the two come to do the same at the
            // same time, and the tensor core waits for both softmaxes (4100 cycles a tile).
#pragma unroll 1
            for (int i = 0; i <= n; ++i) {
              if (i > 0) ready_o(t, kp);
              if (i == 1) o_free();
              wait(bar(S::turn) + 8 * t, turns++ & 1);
              if (i > 0) mma_o(o, t, i == 1, kp);
              if (i < n)
                mma_s(q0 + t * (kChunk >> 4), t, kp, pass);
              else
                pass();
              if (i == n - 1) commit(S::q_empty);
            }
          } else {
            // of a block of one query tile the two take the tiles of tokens in turn, and only give
            // back the others' stages
            const int last = n - 1 - ((n - 1 - t) & 1);  // this one's last tile
            if (last < 0 && !dead) ptx::mbar_arrive(bar(S::q_empty));
#pragma unroll 1
            for (int i = 0; i < n; ++i) {
              if ((i & 1) != t) {
#pragma unroll 1
                for (int u = 0; u < ku + vu; ++u) {
                  wait(bar(S::full) + 8 * kp.st, kp.ph);
                  if (!dead) ptx::mbar_arrive(bar(S::empty) + 8 * kp.st);
                  kp.advance(1);
                }
                continue;
              }
              mma_s(q0, t, kp, stay);
              if (i == last) commit(S::q_empty);
              ready_o(t, kp);
              if (i < 2) o_free();
              mma_o(o, t, i < 2, kp);
            }
            // Without a tile of its own it has not waited for the softmax warps to leave the segment
            // before. It has to: with two phases of o_full behind one another they would wait for the
            // first and take it for one that is still to come.
            if (last < 0) o_free();
          }
          commit(S::o_full + t);
        } else {
          Place<S::NST> vp = kp;
          vp.advance(n > 1 ? 2 * ku : ku);
#pragma unroll 1
          for (int v = -1; v < n; ++v) {
            if (v + 1 < n) {
              mma_s(q0, (tiles + v + 1) & 1, kp, stay);
              if (v >= 0) kp.advance(vu);
              if (v + 2 == n) commit(S::q_empty);
            }
            if (v >= 0) {
              if (v == 0) o_free();
              ready_o((tiles + v) & 1, vp);
              mma_o(tmem + S::o_col, (tiles + v) & 1, v == 0, vp);
              if (v + 2 < n) vp.advance(ku);
            }
          }
          commit(S::o_full);
          tiles += n;
          kp = vp;
        }
      }
      ptx::mma_commit(bar(S::last + t));  // no MMA is in flight when the TMEM goes back
      if (!ptx::mbar_wait(bar(S::last + t), 0, kPrefixWaitNs)) *gave_up = 1;
    }
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    ChunkRecord *rec = places.rec + blockIdx.x;
    rec->gave_up = *gave_up;
    rec->odd = *odd;
  }
  if (*gave_up) {  // copies and MMAs in flight end long before this
    if (tid == 0) atomicOr(a.status, KAMERA_DEVICE_TIMEOUT);
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
  cudaError_t e = cudaFuncGetAttributes(&at, chunk_tc_kernel<S>);
  if (e != cudaSuccess) return e;
  // the warps' shares come out of the registers that the block is launched with
  if (S::kTwo && at.numRegs * S::kThr < S::kRegs) return cudaErrorLaunchOutOfResources;
  return cudaFuncSetAttribute(chunk_tc_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              S::total);
}

template <class S>
cudaError_t launch(const ChunkArgs &a, cudaStream_t s) {
  if (!encode_fn()) return cudaErrorNotSupported;
  Maps m;
  const DevLayout &l = a.lay;
  const int ps = l.page_size, heads = a.hpk < a.shape.rb ? a.hpk : a.shape.rb;
  m.box = ps % kTok == 0 ? kTok : (ps >= 8 && kTok % ps == 0 ? ps : 0);
  const uint32_t box = m.box ? m.box : 8;
  m.copies = kTok / box;
  m.per_page = ps >= kTok ? ps / kTok : 1;
  const long long slots = a.pool.num_slots;
  const __nv_bfloat16 *k = a.pool.k + a.layer * slots * l.row_k;
  const __nv_bfloat16 *v = l.kind == KAMERA_GQA ? a.pool.v + a.layer * slots * l.row_v : k;
  const int vrow = l.kind == KAMERA_GQA ? l.row_v : l.row_k;
  const bool ok =
      encode(&m.k, k, 2, l.row_k, slots, 1, l.row_k, 0, box, 1) &&
      encode(&m.v, v, 2, vrow, slots, 1, vrow, 0, box, 1) &&
      encode(&m.q_block, a.q, 3, a.dk, a.hq, a.n_tokens, a.dk, a.q_stride, heads, a.tb) &&
      encode(&m.q_token, a.q, 3, a.dk, a.hq, a.n_tokens, a.dk, a.q_stride, heads, 1);
  if (!ok) return cudaErrorInvalidValue;
  m.token_bytes = S::DK * 128 * heads;
  m.block_bytes = m.token_bytes * a.tb;
  chunk_tc_kernel<S><<<a.shape.n, S::kThr, S::total, s>>>(a, m);
  return cudaGetLastError();
}

}  // namespace

bool chunk_tc_layout(const DevLayout &l) {
  return (l.kind == KAMERA_GQA && (l.hd == 64 || l.hd == 128)) ||
         (l.kind == KAMERA_MLA && l.latent == 512 && l.rope_d == 64);
}

// Two query tiles: a tile of a block of one of them takes about five sixths of the time of one of two,
// and a block's start and end that of a tile. With tiles alone counted the CTAs of 40 requests, 36 of
// which decode, end at 513000 to 664000 cycles, those of three prompts of 4001 tokens at 449000 to
// 598000, and take 372 and 342 us; with 6, 5 and 6 units 344 and 330, 64-wide heads with a window 73.7
// for 76, but eight requests that decode over 700 tokens, one or two tiles a CTA, 26.2 for 24.6. (4, 3
// and 4: 347, 337, 74.1 and 25.7; a block counted as a tile, tiles alike: 370, 328, 73.8 and 24.8. All
// before the softmax warps met at each segment's start, which takes the prompts to 333.)
// MLA's blocks are alike and have many tiles.
ChunkShape chunk_tc_shape(const DevLayout &l) {
  if (l.kind == KAMERA_MLA) return {kRow, kTokSh, 2, 256, kSms, 1, 1, 0};
  return {2 * kRow, kTokSh, 1, l.hd, kSms, 6, 5, 6};
}

cudaError_t prepare_chunk_tc(const DevLayout &l) {
  if (l.kind == KAMERA_MLA) return configure<Mla512>();
  return l.hd == 128 ? configure<Gqa128>() : configure<Gqa64>();
}

cudaError_t launch_chunk_tc(const ChunkArgs &a, cudaStream_t s) {
  if (a.lay.kind == KAMERA_MLA) return launch<Mla512>(a, s);
  return a.lay.hd == 128 ? launch<Gqa128>(a, s) : launch<Gqa64>(a, s);
}

}  // namespace kamera
