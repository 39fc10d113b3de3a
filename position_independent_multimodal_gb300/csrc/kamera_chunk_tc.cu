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
// Roles: two warpgroups (MLA one) softmax, rescaling and output, a thread to a query row; four warps
// bring K and V rows through the page table into a ring of stages; one thread of the next issues the
// MMAs and the copies of Q. Whole tiles of pages of 8, 16, 32 or 64 slots, or a multiple of 128, come
// as tensor-map copies, one per page and 64 columns; tiles with tokens left out and other page sizes
// as 16-byte cp.async, zero-filled where a token has no slot, so that nothing of a row that no token
// holds is ever multiplied. V of tiles that hold tokens which not all of the block's rows see comes
// through registers: a value that is not finite there would reach rows that do not see it (0 times
// it is no 0), so such blocks are noted and taken again, token by token, by the join kernel.
//   GQA: O and S of two query tiles fill the TMEM. A block of more than 128 rows has two tiles of
//        them that share each K and V tile; of a smaller one (requests that decode) the two take
//        turns with the tiles of tokens, each with a maximum, sum and O of its own, joined at the
//        end. Either way the MMAs of one run during the softmax of the other.
//   MLA: one tile of 128 rows and half of V's columns a CTA (O takes 256 TMEM columns; all 512
//        would leave none for S), S of the next tile issued before P V of this one.
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

// DK, DV: 64-column chunks of K and of the CTA's V columns; QT: tiles of query rows; UC: chunks
// per ring stage; NST: ring stages.
template <int DK_, int DV_, int QT_, int UC_, int NST_>
struct Shape {
  static constexpr int DK = DK_, DV = DV_, QT = QT_, UC = UC_, NST = NST_, NL = 4;
  static constexpr int kSoft = 4 * QT, kMma = kSoft + NL;  // softmax warps; the MMA warp
  // With two query tiles the softmax warps take registers of the others; whole warpgroups
  static constexpr bool kTwo = QT == 2;
  static constexpr int kThr = 32 * (kTwo ? (kMma + 4) / 4 * 4 : kMma + 1);
  static constexpr int kRegsSoft = 160, kRegsRest = 96;
  static constexpr int kRegs = 32 * kSoft * kRegsSoft + (kThr - 32 * kSoft) * kRegsRest;
  static constexpr int kStage = UC * kChunk;
  static constexpr int q = 0;
  static constexpr int ring = QT * DK * kChunk;
  static constexpr int mask = ring + NST * kStage;  // uint32 [kMasks][4]
  static constexpr int xch = mask + kMasks * 16;    // float2 [2][kRow]: maxima and sums
  static constexpr int bar = xch + (kTwo ? 2 * kRow * 8 : 0);
  // mbarriers; those of P: [buffer][half of the tokens]
  static constexpr int full = 0, empty = NST, q_full = empty + NST, q_empty = q_full + 1,
                       s_full = q_empty + 1, p_full = s_full + 2, pv_half = p_full + 4,
                       pv_done = pv_half + 2, o_free = pv_done + 1, o_full = o_free + 1,
                       mk_full = o_full + 2, last = mk_full + kMasks, n_bar = last + 1;
  static constexpr int misc = bar + n_bar * 8;  // TMEM address, give-up flag, odd segments
  static constexpr int scratch = misc + 16;
  static constexpr int total = scratch + sizeof(ChunkScratch<kThr>);
  static constexpr uint32_t o_col = 256;        // O of tile t at o_col + t * 128
  static_assert(total <= 232448, "shared memory of one CTA");
  static_assert(DK % UC == 0 && DV % UC == 0, "whole stages");
  static_assert(kRegs <= 65536 && scratch % 8 == 0, "registers of an SM");
};

using Gqa128 = Shape<2, 2, 2, 2, 5>;
using Gqa64 = Shape<1, 1, 2, 1, 10>;
using Mla512 = Shape<9, 4, 1, 1, 5>;

// Tensor maps of a call: pool rows of the layer (boxes of 64 columns and `box` slots) and query
// rows (64 columns of a block's heads, of all its tokens or of one).
struct Maps {
  CUtensorMap k, v, q_block, q_token;
  int box;                       // slots per copy; 0: rows come by cp.async
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
  int *odd = reinterpret_cast<int *>(smem + S::misc) + 2;  // first and last odd segment
  const ChunkPlaces places = chunk_places(a.shape, a.ws);
  auto bar = [&](int i) { return sb + S::bar + 8 * i; };
  // Waits for a phase, giving up after a.wait_ns or when another thread has. A thread that gave up
  // runs on to its end without waiting, arriving, copying or multiplying: it keeps step with the
  // named barriers only, and no barrier gets an arrival that it does not expect.
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
      ptx::mbar_init(bar(S::p_full + 2 * i), 4);
      ptx::mbar_init(bar(S::p_full + 2 * i + 1), 4);
      ptx::mbar_init(bar(S::pv_half + i), 1);
      ptx::mbar_init(bar(S::o_full + i), 1);
    }
    ptx::mbar_init(bar(S::pv_done), 1);
    ptx::mbar_init(bar(S::o_free), S::kSoft);
    for (int i = 0; i < kMasks; ++i) ptx::mbar_init(bar(S::mk_full + i), S::NL);
    ptx::mbar_init(bar(S::last), 1);
    ptx::fence_mbar_init();
    *gave_up = !begins;
    odd[0] = 0x7FFFFFFF;
    odd[1] = -1;
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
  ChunkWalk walk;
  walk.start(a, st, blockIdx.x);
  ChunkSegment s = {};

  if (warp < S::kSoft) {
    // ---- softmax: thread = query row ----
    if (S::kTwo) ptx::regs_more<S::kRegsSoft>();
    const int w = warp >> 2;                       // query tile
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const float c = fabsf(a.scale) * kLog2e;
    const bool flip = a.scale < 0.f;
    const float inf = __int_as_float(0x7f800000);
    const uint32_t o_t = tmem + S::o_col + w * 128 + lane_off;
    float2 *xch = reinterpret_cast<float2 *>(smem + S::xch);
    auto arrive = [&](uint32_t b) {  // once for the warp
      __syncwarp();
      if (lane == 0 && !dead) ptx::mbar_arrive(b);
    };
    uint32_t mine = 0;   // tiles of this warp so far: phases of its buffers
    uint32_t seen = 0;   // tiles of the CTA's segments so far
    uint32_t segments = 0;
    bool carry = false;
    while (begins && walk.next(a, &s)) {
      if (segments == 0) carry = s.carry;
      const int n = s.t1 - s.t0, rows = s.ntok * s.heads;
      const bool turns = S::kTwo && rows <= kRow;  // the tiles of tokens in turn
      const int i_row = (turns ? 0 : kRow * w) + row;
      const bool live = i_row - lane < rows;  // a warp without rows only keeps step
      int tok, h;
      chunk_row(a, s, i_row < rows ? i_row : 0, &tok, &h);
      // a thread without a row sees all, against a maximum that leaves nothing
      const int see1 = i_row < rows ? s.first + tok + 1 : 0x7FFFFFFF;
      const int see0 = i_row < rows ? first_seen(a, s.first + tok) : 0;
      float m = i_row < rows ? -inf : inf;
      f32x2 la = f2(0.f, 0.f), lb = la;
      int done = 0;  // tiles of this segment
      for (int i = turns ? w : 0; i < n; i += turns ? 2 : 1, ++done, ++mine) {
        const int b = S::kTwo ? w : (mine & 1);
        const uint32_t ph = S::kTwo ? mine & 1 : mine >> 1 & 1;
        wait(bar(S::s_full + b), ph);
        __syncwarp();
        ptx::tc_fence_after();
        if (live) {
          const uint32_t s_t = tmem + b * 128 + lane_off;
          uint32_t xa[32], xb[32];
          ptx::tmem_ld32(s_t, xa);
          // the tile's mask, which is there before S is
          const uint32_t mk = (seen + i) % kMasks;
          wait(bar(S::mk_full + mk), ((seen + i) / kMasks) & 1);
          uint4 msk = *reinterpret_cast<const uint4 *>(smem + S::mask + 16 * mk);
          const int t0 = (s.t0 + i) << kTokSh;
          const bool all = (msk.x & msk.y & msk.z & msk.w) == 0xffffffffu && see0 <= t0 &&
                           see1 - t0 >= kTok && !flip;
          const bool plain = __all_sync(0xffffffffu, all);
          if (!plain) {
            auto seen_of = [&](int k) {  // of 32 tokens, those that the row sees
              const int from = see0 - (t0 + 32 * k), to = see1 - (t0 + 32 * k);
              const uint32_t up = from <= 0 ? 0xffffffffu : from >= 32 ? 0u : 0xffffffffu << from;
              const uint32_t dn = to >= 32 ? 0xffffffffu : to <= 0 ? 0u : (1u << to) - 1u;
              return up & dn;
            };
            msk.x &= seen_of(0);
            msk.y &= seen_of(1);
            msk.z &= seen_of(2);
            msk.w &= seen_of(3);
          }
          const float cs = flip ? -c : c;
          const f32x2 c2 = f2(cs, cs);
          float base = m > -inf ? m * c : 0.f;
          f32x2 ha, hb;         // sums of the weights since they last went into la and lb
          float top, top2;
          uint32_t p[S::kTwo ? 32 : 64];
          // weights of 32 columns in x against `base` into p, their sums, the maximum on the way;
          // two forms: a test of the mask at each weight would cost as much as the weight
          auto weights = [&](const uint32_t *x, uint32_t *to, auto masked, uint32_t bits) {
            const f32x2 nb2 = f2(-base, -base);
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
                hb = add2(hb, f2(p0, p1));
              else
                ha = add2(ha, f2(p0, p1));
              to[e / 2] = pack_bf16(p0, p1);
            }
          };
          auto begin = [&]() {
            ha = hb = f2(0.f, 0.f);
            top = top2 = -inf;
          };
          // Raises the maximum of the rows that want it and rescales what has been summed. `has`: O
          // holds something, and no product into it is in flight.
          auto raise = [&](bool has) {
            const bool first = m == -inf && top > -inf;
            const bool up = first || (top - m) * c > 8.f;
            const float f = up ? (first ? 0.f : exp2_approx((m - top) * c)) : 1.f;
            if (up) m = top;
            base = m > -inf ? m * c : 0.f;
            const f32x2 ff = f2(f, f), zero = f2(0.f, 0.f);
            la = fma2(la, ff, zero);
            lb = fma2(lb, ff, zero);
            if (has) {
#pragma unroll 1
              for (int j = 0; j < S::DV * 4; ++j) {
                uint32_t y[16];
                ptx::tmem_ld16(o_t + 16 * j, y);
                ptx::tmem_ld_wait_all<16>(y);
#pragma unroll
                for (int e = 0; e < 16; ++e) y[e] = __float_as_uint(__uint_as_float(y[e]) * f);
                ptx::tmem_st16(o_t + 16 * j, y);
              }
              ptx::tmem_st_wait();
            }
          };
          auto wants = [&]() {
            top = fmaxf(top, top2);
            return __any_sync(0xffffffffu,
                              (m == -inf && top > -inf) || (top - m) * c > 8.f);
          };
          if constexpr (S::kTwo) {
            // Halves of 64 tokens: the products of the first begin while the second's weights are
            // taken. S of this tile is there, so P V of the tile before is complete.
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
              const uint32_t b0 = hf ? msk.z : msk.x, b1 = hf ? msk.w : msk.y;
              begin();
              ptx::tmem_ld_wait_all<32>(xa);
              ptx::tmem_ld32(s_t + 64 * hf + 32, xb);
              if (plain)
                weights(xa, p, Int<0>(), b0);
              else
                weights(xa, p, Int<1>(), b0);
              ptx::tmem_ld_wait_all<32>(xb);
              if (hf == 0) ptx::tmem_ld32(s_t + 64, xa);
              if (plain)
                weights(xb, p + 16, Int<0>(), b1);
              else
                weights(xb, p + 16, Int<1>(), b1);
              if (wants()) {
                if (hf) {  // the first half's products
                  wait(bar(S::pv_half + w), mine & 1);
                  __syncwarp();
                  ptx::tc_fence_after();
                }
                ptx::tmem_ld_wait_all<32>(xa);
                raise(hf || done > 0);
                begin();
                ptx::tmem_ld32(s_t + 64 * hf, xa);
                ptx::tmem_ld_wait_all<32>(xa);
                weights(xa, p, Int<1>(), b0);
                ptx::tmem_ld32(s_t + 64 * hf + 32, xb);
                ptx::tmem_ld_wait_all<32>(xb);
                weights(xb, p + 16, Int<1>(), b1);
                if (hf == 0) ptx::tmem_ld32(s_t + 64, xa);
              }
              la = add2(la, ha);
              lb = add2(lb, hb);
              ptx::tmem_st32(s_t + 32 * hf, p);  // P over S that has been read
              ptx::tmem_st_wait();
              ptx::tc_fence_before();
              arrive(bar(S::p_full + 2 * b + hf));
            }
          } else {
            auto pass = [&](auto masked) {
              begin();
#pragma unroll
              for (int g = 0; g < 4; ++g) {
                uint32_t *x = g & 1 ? xb : xa, *next = g & 1 ? xa : xb;
                ptx::tmem_ld_wait_all<32>(x);
                if (g < 3) ptx::tmem_ld32(s_t + 32 * (g + 1), next);
                weights(x, p + 16 * g, masked,
                        g == 0 ? msk.x : g == 1 ? msk.y : g == 2 ? msk.z : msk.w);
              }
            };
            if (plain)
              pass(Int<0>());
            else
              pass(Int<1>());
            if (wants()) {
              // P V of the tile before; that of the one before it is complete (this tile's S says
              // so) and this tile's waits for this thread, so the parity is unambiguous
              if (done > 0) {
                wait(bar(S::pv_done), (mine - 1) & 1);
                __syncwarp();
                ptx::tc_fence_after();
              }
              raise(done > 0);
              ptx::tmem_ld32(s_t, xa);
              pass(Int<1>());
            }
            la = add2(la, ha);
            lb = add2(lb, hb);
            ptx::tmem_st32(s_t, p);
            ptx::tmem_st32(s_t + 32, p + 32);
            ptx::tmem_st_wait();
            ptx::tc_fence_before();
            arrive(bar(S::p_full + 2 * b));
          }
        } else {
          ptx::tc_fence_before();
          arrive(bar(S::p_full + 2 * b));
          if (S::kTwo) arrive(bar(S::p_full + 2 * b + 1));
        }
      }
      seen += n;
      // ---- output ----
      wait(bar(S::o_full + w), segments & 1);
      if (turns) wait(bar(S::o_full + (w ^ 1)), segments & 1);
      __syncwarp();
      ptx::tc_fence_after();
      float l;
      {
        float l0, l1;
        f2_split(add2(la, lb), l0, l1);
        l = l0 + l1;
      }
      float f0 = 1.f, f1 = 0.f;  // factors of this warpgroup's O and of the other's
      bool other = false;
      if (turns) {
        xch[w * kRow + row] = make_float2(m, l);
        ptx::barrier_sync(2, 2 * kRow);
        const float2 x = xch[(w ^ 1) * kRow + row];
        const float top = fmaxf(m, x.x);  // (a maximum is never NaN)
        f0 = m == -inf ? 0.f : exp2_approx((m - top) * c);
        f1 = x.x == -inf ? 0.f : exp2_approx((x.x - top) * c);
        other = n > 1 - w;  // it has taken a tile
        l = l * f0 + (other ? x.y * f1 : 0.f);
        m = top;
      }
      if (live) {
        const bool ok = l != 0.f && !*gave_up;
        const float inv = 1.f / l;
        const bool whole = chunk_whole(s);
        const long long rh = (long long)(s.row + tok) * a.hq + h;
        const long long place = (long long)(2 * blockIdx.x + (s.carry ? 0 : 1)) * a.shape.rb + i_row;
        __nv_bfloat16 *out = a.out + rh * a.dv + s.part * a.shape.vw;
        float *part = places.o + place * a.shape.vw;
        const bool write = i_row < rows && !*gave_up;
        // of a row's columns, in turns each warpgroup takes half
        const int cols = S::DV * 64 / (turns ? 2 : 1), from = turns ? w * cols : 0;
        const bool has = !turns || n > w;
        const uint32_t o_other = tmem + S::o_col + lane_off + (w ^ 1) * 128;
        const float g0 = f0 * inv, g1 = f1 * inv;
#pragma unroll 1
        for (int j = from; j < from + cols; j += 32) {
          uint32_t x[32];
          ptx::tmem_ld32(o_t + j, x);
          ptx::tmem_ld_wait_all<32>(x);
#pragma unroll
          for (int e = 0; e < 32; ++e)
            x[e] = ok && has ? __float_as_uint(__uint_as_float(x[e]) * g0) : 0u;
          if (other) {
            uint32_t y[32];
            ptx::tmem_ld32(o_other + j, y);
            ptx::tmem_ld_wait_all<32>(y);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              x[e] = ok ? __float_as_uint(fmaf(__uint_as_float(y[e]), g1, __uint_as_float(x[e])))
                        : 0u;
          }
          if (write && whole) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint4 v;
              v.x = pack_bf16(__uint_as_float(x[e]), __uint_as_float(x[e + 1]));
              v.y = pack_bf16(__uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
              v.z = pack_bf16(__uint_as_float(x[e + 4]), __uint_as_float(x[e + 5]));
              v.w = pack_bf16(__uint_as_float(x[e + 6]), __uint_as_float(x[e + 7]));
              *reinterpret_cast<uint4 *>(out + j + e) = v;
            }
          } else if (write) {
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4 *>(part + j + e) =
                  make_uint4(x[e], x[e + 1], x[e + 2], x[e + 3]);
          }
        }
        if (write && (!turns || w == 0)) {
          const float z = l != 0.f ? (m * c + log2f(l)) * kLn2 : -inf;
          if (!whole)
            places.lse[place] = z;
          else if (s.part == 0)
            a.lse[rh] = z;
        }
      }
      ptx::tc_fence_before();
      arrive(bar(S::o_free));
      ++segments;
    }
    if (tid == 0)
      chunk_note(places.rec + blockIdx.x, s, segments, carry, false, 0x7FFFFFFF, -1);
  } else if (warp < S::kMma) {
    if (S::kTwo) ptx::regs_fewer<S::kRegsRest>();
    // ---- K and V rows into the ring: a warp brings kPart tokens of each tile, a lane holds the
    // slot of one. Copies by tensor map are issued by one thread of the warp, which stands in for
    // the others' arrivals; one issues a copy in about 100 cycles ----
    constexpr int kPart = kTok / S::NL;
    static_assert(kPart == 32, "a lane to a token");
    const int part = warp - S::kSoft, t0 = kPart * part + lane;
    const bool gqa = lay.kind == KAMERA_GQA;
    const __nv_bfloat16 *lk = a.pool.k + (long long)a.layer * a.pool.num_slots * lay.row_k;
    const __nv_bfloat16 *lv =
        gqa ? a.pool.v + (long long)a.layer * a.pool.num_slots * lay.row_v : lk;
    const int vrow = gqa ? lay.row_v : lay.row_k;
    uint32_t *masks = reinterpret_cast<uint32_t *>(smem + S::mask);
    const int piece = lane & 7;  // 16-byte piece of a row
    const int box = maps.box;    // slots of a copy; boxes: copies of this warp per 64 columns
    const int boxes = box == 0 ? 0 : (box <= kPart ? kPart / box : kPart * part % box == 0);
    struct Slots {
      int at;      // this lane's token's
      bool whole;  // every token of the tile is in
    };
    Place<S::NST> at;            // the next stage
    uint32_t tile_no = 0;        // tiles so far
    for (int segment = 0; begins && walk.next(a, &s); ++segment) {
      const int n = s.t1 - s.t0, rows = s.ntok * s.heads;
      const int kcol = gqa ? s.kvh * lay.hd : 0;
      const int vcol = kcol + s.part * a.shape.vw;
      const int lo = first_seen(a, s.first);                 // tokens that a row sees: from here on
      const int all0 = first_seen(a, s.first + s.ntok - 1);  // tokens that all rows see
      const int all1 = s.first + 1;
      auto token = [&](int i) {
        const long long tok = ((long long)(s.t0 + i) << kTokSh) + t0;
        return tok >= lo && tok < s.ctx ? (int)tok : -1;
      };
      int page = 0;  // of the next tile, not looked at yet
      auto load_pages = [&](int i) {
        const int tok = token(i);
        page = tok >= 0 ? load_page(a, s.r, tok) : 0;
      };
      // The next stages: `chunks` chunks from column `col` of a tile's rows
      auto issue = [&](const void *map, const __nv_bfloat16 *base, int row, int col, int chunks,
                       const Slots &sl) {
        if (box && sl.whole) {
          int y[kPart / 8];  // first slots of the copies
#pragma unroll
          for (int k = 0; k < kPart / 8; ++k)
            y[k] = __shfl_sync(0xffffffffu, sl.at, (k * box) & 31);
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
          const __nv_bfloat16 *src = base + col + u * S::UC * 64 + 8 * piece;
#pragma unroll 4
          for (int j = 0; j < kPart / 4; ++j) {  // four of this warp's tokens at a time
            const int q = 4 * j + (lane >> 3), t = kPart * part + q;
            const int slot = __shfl_sync(0xffffffffu, sl.at, q);
            const __nv_bfloat16 *p = slot >= 0 ? src + (long long)slot * row : a.pool.k;
#pragma unroll
            for (int k = 0; k < S::UC; ++k)
              ptx::cp_async16(dst + k * kChunk + t * 128 + ((piece ^ (t & 7)) << 4),
                              slot >= 0 ? p + k * 64 : p, slot >= 0 ? 16u : 0u);
          }
          ptx::cp_async_mbar_arrive(full);
        }
      };
      // V of a tile with tokens that not all rows see, through registers
      auto issue_v_looked_at = [&](int i, const Slots &sl) {
        bool found = false;
        for (int u = 0; u < S::DV / S::UC; ++u) {
          const uint32_t dst = S::ring + at.st * S::kStage, full = bar(S::full) + 8 * at.st;
          wait(bar(S::empty) + 8 * at.st, at.ph ^ 1);
          at.advance(1);
          if (__any_sync(0xffffffffu, dead)) {
            dead = true;
            continue;
          }
          const __nv_bfloat16 *src = lv + vcol + u * S::UC * 64 + 8 * piece;
#pragma unroll 1
          for (int j0 = 0; j0 < kPart / 4; j0 += 4) {
            uint4 v[4][S::UC];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int slot = __shfl_sync(0xffffffffu, sl.at, 4 * (j0 + j) + (lane >> 3));
#pragma unroll
              for (int k = 0; k < S::UC; ++k)
                v[j][k] = slot >= 0 ? __ldg(reinterpret_cast<const uint4 *>(
                                          src + (long long)slot * vrow + k * 64))
                                    : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int t = kPart * part + 4 * (j0 + j) + (lane >> 3);
              const int tok = ((s.t0 + i) << kTokSh) + t;
#pragma unroll
              for (int k = 0; k < S::UC; ++k) {
                found |= (tok < all0 || tok >= all1) && odd8(v[j][k]);
                *reinterpret_cast<uint4 *>(smem + dst + k * kChunk + t * 128 +
                                           ((piece ^ (t & 7)) << 4)) = v[j][k];
              }
            }
          }
          ptx::fence_proxy_async_smem();
          ptx::mbar_arrive(full);
        }
        if (found) {
          atomicMin(odd, segment);
          atomicMax(odd + 1, segment);
        }
      };
      Slots kt;  // of the last K tile
      auto load_k = [&](int i) {
        const int mk = tile_no++ % kMasks, tok = token(i);
        kt.at = tok >= 0 ? slot_in(a, page, tok) : -1;
        const uint32_t bits = __ballot_sync(0xffffffffu, kt.at >= 0);
        if (i + 1 < n) load_pages(i + 1);  // ahead of its use
        if (lane == 0) {
          masks[4 * mk + part] = bits;
          if (!dead) ptx::mbar_arrive(bar(S::mk_full) + 8 * mk);
        }
        __syncwarp();
        ptx::barrier_sync(1, 32 * S::NL);
        const uint4 m = *reinterpret_cast<const uint4 *>(masks + 4 * mk);
        kt.whole = (m.x & m.y & m.z & m.w) == 0xffffffffu;
        issue(&maps.k, lk, lay.row_k, kcol, S::DK, kt);
      };
      auto load_v = [&](int i, const Slots &sl) {
        const long long tok = (long long)(s.t0 + i) << kTokSh;
        const long long end = min(tok + kTok, (long long)s.ctx), from = max(tok, (long long)lo);
        if (from < min(end, (long long)all0) || max(from, (long long)all1) < end)
          issue_v_looked_at(i, sl);
        else
          issue(&maps.v, lv, vrow, vcol, S::DV, sl);
      };
      // the stages come in the order in which they are read: two query tiles K0 V0 K1 V1 ..., one
      // K0 K1 V0 K2 V1 ... V(n-1)
      const int ahead = S::kTwo && rows > kRow ? 1 : 2;
      load_pages(0);
      load_k(0);
      Slots vt = kt;  // of the next V tile
      if (ahead == 2 && n > 1) load_k(1);
      for (int i = 0; i < n; ++i) {
        const Slots next = kt;
        load_v(i, vt);
        if (i + ahead < n) load_k(i + ahead);
        vt = ahead == 1 ? kt : next;
      }
    }
    ptx::cp_async_wait_all();
  } else {
    if (S::kTwo) ptx::regs_fewer<S::kRegsRest>();
    // ---- MMAs and Q, one thread. Issuing an MMA takes a few instructions only: the descriptors of
    // a tile's steps differ by constants ----
    if (warp == S::kMma && ptx::elect_one()) {
      uint32_t segs = 0;
      constexpr uint32_t id_s =
          1u << 4 | 1u << 7 | 1u << 10 | (kTok >> 3) << 17 | (kRow >> 4) << 24;
      // V is MN-major
      constexpr uint32_t id_o =
          1u << 4 | 1u << 7 | 1u << 10 | 1u << 16 | (S::UC * 64 >> 3) << 17 | (kRow >> 4) << 24;
      constexpr int ku = S::DK / S::UC, vu = S::DV / S::UC;  // stages of a K and a V tile
      const uint32_t ring = sb + S::ring;
      Place<S::NST> kp, vp;
      uint32_t tiles = 0;                                // one query tile: k has S buffer k % 2
      uint32_t p_ph = 0;                                 // a bit for each S buffer
      const uint32_t q0 = desc_k(sb + S::q);             // [chunk][query tile][128 rows]
      auto landed = [&](const Place<S::NST> &at) {
        wait(bar(S::full) + 8 * at.st, at.ph);
        ptx::fence_proxy_async_smem();
      };
      // S of query tile t into TMEM buffer b against the K tile at kp; ends: bit 0 the first,
      // bit 1 the last reader of its stages
      auto mma_s = [&](int t, uint32_t b, auto ends) {
        const uint32_t d = tmem + b * 128, qt = q0 + t * (kChunk >> 4);
        Place<S::NST> at = kp;
#pragma unroll
        for (int u = 0; u < ku; ++u) {
          if (ends.v & 1) landed(at);
          if (dead) return;
          const uint32_t k = desc_k(ring + at.st * S::kStage);
#pragma unroll
          for (int x = 0; x < S::UC * 4; ++x)
            ptx::mma_bf16(
                d, desc(qt + (((u * S::UC + (x >> 2)) * S::QT * kChunk + (x & 3) * 32) >> 4)),
                desc(k + (((x >> 2) * kChunk + (x & 3) * 32) >> 4)), id_s, (u | x) ? 1u : 0u);
          if (ends.v & 2) ptx::mma_commit(bar(S::empty) + 8 * at.st);
          at.advance(1);
        }
        ptx::mma_commit(bar(S::s_full) + 8 * b);
        if (ends.v & 2) kp = at;
      };
      // O of tile t (+)= P in buffer b times the V tile at vp
      auto mma_o = [&](int t, uint32_t b, bool first_tile, auto ends) {
        const uint32_t p = tmem + b * 128, d = tmem + S::o_col + t * 128;
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
            if (S::kTwo && x == kTok / 32) {
              ptx::mma_commit(bar(S::pv_half) + 8 * t);
              wait(bar(S::p_full) + 16 * b + 8, (p_ph >> b) & 1);
              if (dead) return;
              ptx::tc_fence_after();
            }
            ptx::mma_bf16_ta(d + u * S::UC * 64, p + 8 * x, desc(v + x * (2048 >> 4)), id_o,
                             x ? 1u : (first_tile ? 0u : 1u));
          }
          if (ends.v & 2) ptx::mma_commit(bar(S::empty) + 8 * at.st);
          at.advance(1);
        }
        p_ph ^= 1u << b;
        if (!S::kTwo) ptx::mma_commit(bar(S::pv_done));
        if (ends.v & 2) vp = at;
      };
      auto o_free = [&]() {  // O of the segment before has been read
        if (segs) wait(bar(S::o_free), (segs - 1) & 1);
      };
      auto commit = [&](int b) {
        if (!dead) ptx::mma_commit(bar(b));
      };
      constexpr Int<1> first;
      constexpr Int<2> last;
      constexpr Int<3> only;
      while (begins && walk.next(a, &s)) {
        const int n = s.t1 - s.t0;
        // Q, once S of the segment before is complete. Rows of a copy past the block's are other
        // tokens' or zero: their results go nowhere
        if (segs) wait(bar(S::q_empty), (segs - 1) & 1);
        if (!dead) {
          const bool one = s.ntok == 1;
          ptx::mbar_arrive_expect_tx(bar(S::q_full), one ? maps.token_bytes : maps.block_bytes);
          for (int c = 0; c < S::DK; ++c)
            ptx::tma_3d(sb + S::q + c * S::QT * kChunk, one ? &maps.q_token : &maps.q_block, c * 64,
                        s.h0, s.row, bar(S::q_full));
        }
        wait(bar(S::q_full), segs & 1);
        ptx::fence_proxy_async_smem();
        vp = kp;
        if constexpr (S::kTwo) {
          if (s.ntok * s.heads > kRow) {
            vp.advance(ku);
            mma_s(0, 0, first);
            mma_s(1, 1, last);
            o_free();
            for (int i = 0; i + 1 < n; ++i) {
              kp.advance(vu);
              mma_o(0, 0, i == 0, first);
              mma_s(0, 0, first);
              mma_o(1, 1, i == 0, last);
              mma_s(1, 1, last);
              vp.advance(ku);
            }
            commit(S::q_empty);
            mma_o(0, 0, n == 1, first);
            commit(S::o_full);
            mma_o(1, 1, n == 1, last);
            commit(S::o_full + 1);
          } else {
            vp.advance(n > 1 ? 2 * ku : ku);
            mma_s(0, 0, only);
            if (n > 1) mma_s(0, 1, only);
            o_free();
            for (int i = 0; i < n; ++i) {
              if (i + 2 == n || n == 1) commit(S::q_empty);
              mma_o(i & 1, i & 1, i < 2, only);
              if (i + 2 < n) {
                kp.advance(vu);
                mma_s(0, i & 1, only);
                vp.advance(ku);
              }
            }
            commit(S::o_full);
            commit(S::o_full + 1);
          }
        } else {
          vp.advance(n > 1 ? 2 * ku : ku);
          mma_s(0, tiles & 1, only);
          if (n == 1) commit(S::q_empty);
          for (int i = 0; i < n; ++i) {
            if (i + 1 < n) {
              if (i > 0) kp.advance(vu);
              mma_s(0, (tiles + i + 1) & 1, only);
              if (i + 2 == n) commit(S::q_empty);
            }
            if (i == 0) o_free();
            mma_o(0, (tiles + i) & 1, i == 0, only);
            if (i + 2 < n) vp.advance(ku);
          }
          commit(S::o_full);
          tiles += n;
        }
        kp = vp;  // the segment's end
        ++segs;
      }
      ptx::mma_commit(bar(S::last));  // no MMA is in flight when the TMEM goes back
      if (!ptx::mbar_wait(bar(S::last), 0, kPrefixWaitNs)) *gave_up = 1;
    }
    __syncwarp();
  }
  ptx::tc_fence_before();
  __syncthreads();
  if (tid == 0) {
    ChunkRecord *rec = places.rec + blockIdx.x;
    rec->gave_up = *gave_up;
    rec->odd0 = odd[0];
    rec->odd1 = odd[1];
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

ChunkShape chunk_tc_shape(const DevLayout &l) {
  if (l.kind == KAMERA_MLA) return {kRow, kTokSh, 2, 256, kSms};
  return {2 * kRow, kTokSh, 1, l.hd, kSms};
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
