// Attention masses on the tensor cores: GQA with head_dim 64 or 128, MLA with a latent of 512 and a
// rope band of 64. One persistent CTA per SM works its share of units off (kamera_mass.cuh).
//
//   S^T [128 cached tokens x 128 query rows] = K Q^T     tcgen05, K and Q from shared memory
//   mass_u += sum over the columns of 2^(c S - c' lse),  c = scale log2 e,  c' = log2 e
//
// The transposed product leaves a cached token to a thread (of each part of the columns), so its sum
// stays in a register over all query rows of a block and no two threads add to one number. K rows of
// a block stay in shared memory while the query rows of a KV head pass through a ring; S has two
// buffers a tile (MLA four, for pieces of its sums), so products and weights never wait for one another
// but where one is slower: 32768 weights a unit take the special-function units 1024 cycles, the
// products of two tiles 1040.
//
// Roles: sixteen warps take weights (GQA: two tiles of 128 tokens, two parts of 64 columns; MLA: one
// tile, four parts of 32), one brings K (and GQA's Q; MLA's has a warp of its own, as each of its units
// takes nine stages of Q), one the rows' log-sum-exps, and a thread for each tile of tokens issues the
// MMAs. Copies of K as in kamera_chunk_tc.cu.
//
// Measured: 32 requests that decode over 3000 to 6001 tokens (28 query heads, 4 KV heads of 128) in 41
// us, 3.6 TB/s of K; 250 new tokens over 30000 in 61.5 us, 1730 weights a clock of the chip's 4860. The
// weights' warps have 184 instructions for 64 weights and some 150 more around them; tokens next to
// the new ones, whose columns are seen in part, take longer, and the CTA that has them ends last.
#include "kamera_mass.cuh"
#include "kamera_ptx.cuh"
#include "kamera_smem.cuh"
#include "kamera_tc.cuh"

namespace kamera {

namespace {

constexpr int kTokSh = 7, kTok = 1 << kTokSh;  // tokens of an MMA
constexpr int kRow = 128;                      // query rows of a tile
constexpr int kSegs = 8;                       // segments that are kept
constexpr int kZ = 2;                          // tiles of query rows whose log-sum-exps are kept

// A segment, as the roles share it.
struct Seg {
  int row, n, past, ctx;  // of the request: first row of q, new tokens, tokens before them, context
  int r, tok0;            // the request, the block's first token
  int i0, ni, k0, k1;     // its tiles of new tokens, its units; k0 == k1: there are no more
  int more;               // -1: starts inside its block; else workers that follow on it
};

// DK: 64-column chunks of K; KT: tiles of 128 tokens; SETS: sets of K tiles; UC: chunks of a stage of
// Q; NST: stages of Q; AC: chunks that a score is summed over in TMEM. The tensor core cuts its sums
// off where it should round them, so each of its steps takes a little of a score's size: 8e-8 of it
// over the 8 steps of 128 columns, 4.3e-7 over the 36 of MLA, where weights of large scores come out
// 4e-6 too small. There the sum is taken in pieces, which take four TMEM buffers in turn and are added
// in registers, rounded. Measured over six requests of 100 new tokens over 5000 (the masses' error, the
// time): in one piece 3.8e-6, 47 us; pieces of three chunks 1.2e-6, 48; of two 8.5e-7, 49; of one
// 5.5e-7, 51 us. Products in float32 with rounded sums give 7e-7: a chunk a piece it is.
template <int DK_, int KT_, int SETS_, int UC_, int NST_, int AC_>
struct Shape {
  static constexpr int DK = DK_, KT = KT_, SETS = SETS_, UC = UC_, NST = NST_, AC = AC_;
  static constexpr int kPieces = (DK + AC - 1) / AC;  // pieces of a sum
  static constexpr int kBuf = 4 / KT;                 // TMEM buffers of a tile
  static constexpr int kSoft = 16, kLoad = 16, kLse = 17, kMma = 18;
  // (one tile of tokens takes more of Q than of K: a warp of its own brings it)
  static constexpr int kQ = KT == 1 ? kMma + KT : kLoad;
  static constexpr int kThr = 32 * (KT == 1 ? kQ + 1 : kMma + KT);
  static constexpr int kParts = 4 / KT, kCols = kRow / kParts;  // parts of the columns, columns of one
  static constexpr int kStage = UC * kChunk, kSet = DK * KT * kChunk;
  static constexpr int k = 0;                        // [set][chunk][tile][128 rows]
  static constexpr int ring = k + SETS * kSet;
  static constexpr int z = ring + NST * kStage;      // float [kZ][kRow]: c' lse, inf for no row
  static constexpr int xch = z + kZ * kRow * 4;      // float [kParts - 1][KT * kTok]: sums
  // int [kZ][4] of a unit: its rows; how tile 0 and tile 1 are taken (0: all rows see the tile's
  // tokens; 1: a run of them each token; 2: and their log-sum-exps are to be looked at); its first of
  // its request's new tokens
  static constexpr int flags = xch + (kParts - 1) * KT * kTok * 4;
  static constexpr int bar = flags + kZ * 16;
  static constexpr int k_full = 0, k_empty = k_full + SETS * DK, q_full = k_empty + SETS * DK,
                       q_empty = q_full + NST, s_full = q_empty + NST, s_free = s_full + kBuf * KT,
                       z_full = s_free + kBuf * KT, z_free = z_full + kZ, sg_full = z_free + kZ,
                       last = sg_full + kSegs, n_bar = last + KT;
  static constexpr int misc = bar + n_bar * 8;       // TMEM address, give-up flag
  static constexpr int walk = misc + 16;
  static constexpr int seg = walk + (sizeof(MassWalk) + 15) / 16 * 16;
  static constexpr int total = seg + kSegs * sizeof(Seg);
  static constexpr int scratch = z;                  // of the start
  static_assert(total <= 232448, "shared memory of one CTA");
  static_assert(DK % UC == 0 && AC % UC == 0, "whole stages");
  static_assert(walk % 8 == 0 && scratch % 8 == 0 && flags % 16 == 0, "of wide loads and stores");
  static_assert(kPieces == 1 || kCols == 32, "a piece's columns in registers");
  static_assert(sizeof(ChunkScratch<kThr>) <= kZ * kRow * 4, "the start's scratch");
};

using Gqa128 = Shape<2, 2, 2, 2, 3, 2>;
using Gqa64 = Shape<1, 2, 3, 1, 4, 1>;
using Mla512 = Shape<9, 1, 1, 1, 4, 1>;

struct Maps {
  CUtensorMap k, q_block, q_token;
  int box, copies, per_page;     // as in kamera_chunk_tc.cu
  int block_bytes, token_bytes;  // of a chunk of the query copies
};

template <class S>
__global__ void __launch_bounds__(S::kThr, 1) mass_tc_kernel(const __grid_constant__ MassArgs a,
                                                             const __grid_constant__ Maps maps) {
  extern __shared__ __align__(1024) unsigned char smem[];
  const uint32_t sb = ptx::smem_addr(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const ChunkArgs &b = a.b;
  const DevLayout &lay = b.lay;
  volatile uint32_t *misc = reinterpret_cast<volatile uint32_t *>(smem + S::misc);
  volatile uint32_t *gave_up = misc + 1;
  const MassPlaces places = mass_places(a.shape, a.ws);
  auto bar = [&](int i) { return sb + S::bar + 8 * i; };
  // Waits for a phase, giving up after b.wait_ns or when another thread has. A thread that gave up
  // runs on to the end of its segment without waiting, arriving, copying or multiplying: it keeps step
  // with the named barriers only, and no barrier gets an arrival that it does not expect. Threads that
  // meet (a warp, the warps of a token's parts) leave together.
  bool dead = false;
  auto wait = [&](uint32_t at, uint32_t parity) {
    if (__builtin_expect(dead || ptx::mbar_try_wait(at, parity), 1)) return;
    const uint64_t t0 = ptx::globaltimer();
    while (!ptx::mbar_try_wait_for(at, parity, 20000)) {
      if (*gave_up || ptx::globaltimer() - t0 > b.wait_ns) {
        *gave_up = 1;
        dead = true;
        return;
      }
    }
  };

  // The swizzled layouts want 1024-byte groups (there is no static memory here, so they get them);
  // without them, or without time to wait, nothing is begun and the kernel ends as if it gave up.
  const bool begins = (sb & 1023u) == 0 && b.wait_ns != 0;
  if (warp == S::kMma) {
    ptx::tmem_alloc(sb + S::misc, 512);
    ptx::tmem_relinquish();
  }
  if (tid == 0) {
    for (int i = 0; i < S::SETS * S::DK; ++i) {
      ptx::mbar_init(bar(S::k_full + i), 32);
      ptx::mbar_init(bar(S::k_empty + i), S::KT);
    }
    for (int i = 0; i < S::NST; ++i) {
      ptx::mbar_init(bar(S::q_full + i), 1);
      ptx::mbar_init(bar(S::q_empty + i), S::KT);
    }
    for (int i = 0; i < S::kBuf * S::KT; ++i) {
      ptx::mbar_init(bar(S::s_full + i), 1);
      ptx::mbar_init(bar(S::s_free + i), S::kSoft / S::KT);
    }
    for (int i = 0; i < kZ; ++i) {
      ptx::mbar_init(bar(S::z_full + i), 1);
      ptx::mbar_init(bar(S::z_free + i), S::kSoft);
    }
    for (int i = 0; i < kSegs; ++i) ptx::mbar_init(bar(S::sg_full + i), 1);
    for (int i = 0; i < S::KT; ++i) ptx::mbar_init(bar(S::last + i), 1);
    ptx::fence_mbar_init();
    *gave_up = !begins;
    ptx::prefetch_map(&maps.k);
    ptx::prefetch_map(&maps.q_block);
    ptx::prefetch_map(&maps.q_token);
  }
  // rows of a stage that no copy of a whole tile of query rows writes stay 0: their scores are finite
  for (int i = tid; i < S::NST * S::kStage / 16; i += S::kThr)
    reinterpret_cast<uint4 *>(smem + S::ring)[i] = make_uint4(0, 0, 0, 0);
  ptx::fence_proxy_async_smem();
  const ChunkStart st = mass_start<S::kThr>(
      a, blockIdx.x, reinterpret_cast<ChunkScratch<S::kThr> *>(smem + S::scratch));
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = misc[0];
  ptx::launch_dependents();

  // The worker's segments. The loading warp walks them and publishes each after the first unit of the
  // one before; one with no units ends them. With kSegs places the one that is overwritten has been
  // left by all: the loader is at most NST units ahead of the products, those two of the weights.
  MassWalk *walk = reinterpret_cast<MassWalk *>(smem + S::walk);
  Seg *segs = reinterpret_cast<Seg *>(smem + S::seg);
  uint32_t seg_no = 0;  // segments taken
  auto take_segment = [&]() -> const Seg * {  // the next one, null behind the last
    const uint32_t k = seg_no % kSegs;
    wait(bar(S::sg_full) + 8 * k, seg_no / kSegs & 1);
    const Seg *s = segs + k;
    if (dead || s->k0 == s->k1) return nullptr;
    ++seg_no;
    return s;
  };
  // The same for a whole warp: of its threads one alone may have given up (the elected one, on a stage),
  // and none may leave while the others go on to what they do together.
  auto take_whole = [&]() -> const Seg * {
    const Seg *s = take_segment();
    dead = __any_sync(0xffffffffu, dead);
    return dead ? nullptr : s;
  };
  // Calls f(unit so far, KV head, piece of its query heads, tile of new tokens, first unit of the KV
  // head's K rows, last one) for the units of a segment.
  uint32_t units = 0;
  auto each_unit = [&](const Seg *s, auto f) {
    const int ni = s->ni, i0 = s->i0, k1 = s->k1;
    int hp = s->k0 / ni, i = s->k0 - hp * ni;
    int kvh = hp / b.pieces, piece = hp - kvh * b.pieces;
    bool first = true;
#pragma unroll 1
    for (int k = s->k0; k < k1; ++k, ++units) {
      const bool ends = i + 1 == ni, last = k + 1 == k1 || (ends && piece + 1 == b.pieces);
      f(units, kvh, piece, i0 + i, first, last);
      first = last;
      if (ends) {
        i = 0;
        if (++piece == b.pieces) {
          piece = 0;
          ++kvh;
        }
      } else {
        ++i;
      }
    }
  };
  if (warp == S::kLoad) {
    MassWalk w;
    w.start(a, st, blockIdx.x);
    if (!begins) w.left = 0;
    if (lane == 0) *walk = w;
    __syncwarp();
  }

  if (warp < S::kSoft) {
    // ---- weights: a thread to a token and a part of the columns ----
    constexpr int kPer = S::kSoft / S::KT;           // warps of a tile
    const int w = warp / kPer, part = warp % kPer >> 2;
    const int quarter = warp & 3, mine = w * kTok + quarter * 32 + lane;  // the token in the block
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    const float c = b.scale * kLog2e, inf = __int_as_float(0x7f800000);
    const uint32_t nothing = c < 0.f ? 0x7f800000u : 0xff800000u;  // a score of no weight
    const int group = 1 + w * 4 + quarter;           // named barrier of the tokens' warps
    float *xch = reinterpret_cast<float *>(smem + S::xch);
    auto arrive = [&](uint32_t at) {  // once for the warp
      __syncwarp();
      if (lane == 0 && !dead) ptx::mbar_arrive(at);
    };
    MassRecord rec = {0, 0, 0, 0, 0, {0, 0, 0}};
    // The warps of a token's parts meet at a barrier in every segment, so they leave together. Then all
    // of them have read the sums of the segment before, too, which the next one's are written over.
    auto take_together = [&]() -> const Seg * {
      const Seg *s = take_segment();
      return ptx::barrier_or(group, 32 * S::kParts, dead) ? nullptr : s;
    };
    while (const Seg *sp = take_together()) {
      const int tok = sp->tok0 + mine, ctx = sp->ctx, past = sp->past, more = sp->more, r = sp->r;
      rec.head = more > 0;
      rec.more = more;
      rec.r = r;
      rec.tok0 = sp->tok0;
      bool have = false;  // the token has a slot
      if (part == 0 && tok < ctx && tok >= first_seen(b, past + sp->i0 * b.tb)) {
        const int page = load_page(b, r, tok);
        have = page >= 0 && ((long long)page + 1) * lay.page_size <= b.pool.num_slots;
      }
      f32x2 sa = f2(0.f, 0.f), sc = sa;
      // (what a unit is comes with its log-sum-exps: these warps have no instructions to spare)
      const uint32_t end = units + (sp->k1 - sp->k0);
#pragma unroll 1
      for (; units != end; ++units) {
        const uint32_t u = units, zs = u % kZ;
        wait(bar(S::z_full) + 8 * zs, u / kZ & 1);
        __syncwarp();  // (all take the same flags, also where they gave up)
        const int4 flags = *reinterpret_cast<const int4 *>(smem + S::flags + 16 * zs);
        const int rows = flags.x, how = w ? flags.z : flags.y;
        int see0 = 0, see1 = rows;  // the columns whose tokens see this one: [see0, see1)
        if (how) {
          const int ahead = tok - past - flags.w;
          see0 = ahead > 0 ? min(ahead, kRow) * b.hpk : 0;
          see1 = min(rows, b.window > 0 && ahead < kRow - b.window ? max(ahead + b.window, 0) * b.hpk
                                                                   : kRow);
        }
        const float *z = reinterpret_cast<const float *>(smem + S::z) + zs * kRow + part * S::kCols;
        // the weights of 16 columns from g on, all of which are seen
        auto some = [&](const uint32_t *x, int g) {
#pragma unroll
          for (int e = 0; e < 16; e += 4) {
            const float4 z4 = *reinterpret_cast<const float4 *>(z + g + e);
            const float p0 = exp2_approx(fmaf(__uint_as_float(x[e]), c, -z4.x));
            const float p1 = exp2_approx(fmaf(__uint_as_float(x[e + 1]), c, -z4.y));
            const float p2 = exp2_approx(fmaf(__uint_as_float(x[e + 2]), c, -z4.z));
            const float p3 = exp2_approx(fmaf(__uint_as_float(x[e + 3]), c, -z4.w));
            sa = add2(sa, f2(p0, p1));
            sc = add2(sc, f2(p2, p3));
          }
        };
        // the weights of 32 columns
        auto weigh = [&](uint32_t *x, int g) {
          const int col0 = part * S::kCols + g;
          if (__builtin_expect(how == 2, 0)) {
            float s0 = 0.f;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const bool on = col0 + e >= see0 && col0 + e < see1 && z[g + e] != inf;
              s0 += on ? exp2_approx(fmaf(__uint_as_float(x[e]), c, -z[g + e])) : 0.f;
            }
            sa = add2(sa, f2(s0, 0.f));
            return;
          }
          // (columns behind the rows too: of a key with an infinity they are 0 times it, NaN)
          if (how == 1 || col0 + 32 > rows) {
            const int from = see0 - col0, to = see1 - col0;
            const uint32_t up = from <= 0 ? 0xffffffffu : from >= 32 ? 0u : 0xffffffffu << from;
            const uint32_t dn = to >= 32 ? 0xffffffffu : to <= 0 ? 0u : (1u << to) - 1u;
            const uint32_t seen = up & dn;
            if (__all_sync(0xffffffffu, seen == 0)) return;
            if (!__all_sync(0xffffffffu, seen == 0xffffffffu)) {
#pragma unroll
              for (int e = 0; e < 32; ++e) x[e] = seen & (1u << e) ? x[e] : nothing;
            }
          }
          some(x, g);
          some(x + 16, g + 16);
        };
        // S of buffer n, of this unit or a piece of its sum
        auto take = [&](uint32_t n) {
          wait(bar(S::s_full + w * S::kBuf) + 8 * (n % S::kBuf), n / S::kBuf & 1);
          __syncwarp();
          ptx::tc_fence_after();
          return tmem + (w * S::kBuf + n % S::kBuf) * 128 + part * S::kCols + lane_off;
        };
        auto give = [&](uint32_t n) {
          ptx::tc_fence_before();
          arrive(bar(S::s_free + w * S::kBuf) + 8 * (n % S::kBuf));
        };
        const int cols = rows - part * S::kCols;  // that this part has
        if constexpr (S::kPieces == 1) {
          const uint32_t at = take(u);
          if (how == 0 && cols > S::kCols - 16) {
            // S comes sixteen columns ahead of the weights, and its buffer goes back before the last
            uint32_t x[2][16];
            ptx::tmem_ld16(at, x[0]);
            ptx::tmem_ld_wait_all<16>(x[0]);
#pragma unroll
            for (int g = 0; g < S::kCols; g += 16) {
              uint32_t *next = x[(g >> 4 & 1) ^ 1];
              if (g + 16 < S::kCols) {
                ptx::tmem_ld16(at + g + 16, next);
              } else {
                give(u);
                uint32_t *y = x[g >> 4 & 1];
                // as in weigh, four columns at a time (4 x 250 over 30000: 150 us, 154 with all sixteen
                // looked at, 148 with none)
#pragma unroll
                for (int q = 16; q > 0; q -= 4) {
                  if (g + q <= cols) break;
#pragma unroll
                  for (int e = q - 4; e < q; ++e) y[e] = g + e < cols ? y[e] : nothing;
                }
              }
              some(x[g >> 4 & 1], g);
              if (g + 16 < S::kCols) ptx::tmem_ld_wait_all<16>(next);
            }
          } else {
#pragma unroll 1
            for (int g = 0; g < S::kCols && g < cols; g += 32) {
              uint32_t x[32];
              ptx::tmem_ld32(at + g, x);
              ptx::tmem_ld_wait_all<32>(x);
              weigh(x, g);
            }
            give(u);
          }
        } else {
          uint32_t x[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = 0;
#pragma unroll 1
          for (int k = 0; k < S::kPieces; ++k) {
            const uint32_t n = u * S::kPieces + k, at = take(n);
            if (cols > 0) {
              uint32_t y[32];
              ptx::tmem_ld32(at, y);
              ptx::tmem_ld_wait_all<32>(y);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                x[e] = __float_as_uint(__uint_as_float(x[e]) + __uint_as_float(y[e]));
            }
            give(n);
          }
          if (cols > 0) weigh(x, 0);
        }
        arrive(bar(S::z_free) + 8 * zs);  // (all lanes have read theirs)
      }
      float sum;
      {
        float s0, s1;
        f2_split(add2(sa, sc), s0, s1);
        sum = s0 + s1;
      }
      if (part > 0) xch[(part - 1) * (S::KT * kTok) + mine] = sum;
      ptx::barrier_sync(group, 32 * S::kParts);
      if (part == 0) {
#pragma unroll
        for (int k = 0; k + 1 < S::kParts; ++k) sum += xch[k * (S::KT * kTok) + mine];
        sum = have ? sum : 0.f;
        if (!*gave_up) {
          if (more != 0) {
            places.sum[(2ll * blockIdx.x + (more < 0 ? 0 : 1)) * a.shape.kt + mine] = sum;
          } else if (tok < ctx) {
            float *m = a.mass + (long long)r * a.mass_stride + tok;
            *m = a.decay == 0.f ? sum : fmaf(a.decay, *m, sum);
          }
        }
      }
    }
    if (tid == 0) places.rec[blockIdx.x] = rec;
  } else if (warp == S::kLoad || warp == S::kQ) {
    // ---- K and Q into shared memory. K comes as copies by tensor map, a lane to a page, or for page
    // sizes that are no box of one piece by piece. What is in the rows of tokens that no one sees, or
    // that have no slot, does not matter: a row of S^T is a token's own, and theirs are left out ----
    const bool gqa = lay.kind == KAMERA_GQA;
    const int box = maps.box, each = maps.copies, per_page = maps.per_page;
    const unsigned pages = (unsigned)(b.pool.num_slots / lay.page_size);
    uint32_t sets = 0, stages = 0, published = 0;
    auto publish = [&]() {  // the next segment
      if (warp == S::kLoad && lane == 0) {
        Seg *to = segs + published % kSegs;
        MassSegment m;
        if (walk->next(a, &m)) {
          *to = {m.q.row, m.q.n, m.q.past, m.q.ctx, m.r, m.tok0, m.i0, m.ni, m.k0, m.k1,
                 m.carry ? -1 : m.more};
        } else {
          to->k0 = to->k1 = 0;
        }
        if (!dead) ptx::mbar_arrive(bar(S::sg_full) + 8 * (published % kSegs));
      }
      ++published;
      __syncwarp();
    };
    // Of a segment: the first slot of the lane's copy (tile lane / copies, its page), -1 where none of
    // its tokens is looked at or the page is outside the pool
    auto look_up = [&](const Seg *sp) {
      if (warp != S::kLoad || sp->k0 == sp->k1 || !box || lane >= each * S::KT) return -1;
      const long long tok = sp->tok0 + (long long)lane * box;
      if (tok + box <= first_seen(b, sp->past + sp->i0 * b.tb) || tok >= sp->ctx) return -1;
      const int t = (int)(tok >> kTokSh);
      const int entry = __ldg(b.pool.pt + (long long)sp->r * b.pool.pt_stride +
                              (each == 1 ? t / per_page : t * each + lane % each));
      if ((unsigned)entry < pages)
        return entry * lay.page_size + (each == 1 ? t % per_page * kTok : 0);
      atomicOr(b.status, KAMERA_DEVICE_SLOT_OOB);
      return -1;
    };
    publish();
    wait(bar(S::sg_full), 0);
    int next_y = look_up(segs);
    while (const Seg *sp = take_whole()) {
      const int tok0 = sp->tok0, ctx = sp->ctx, r = sp->r;
      const int lo = first_seen(b, sp->past + sp->i0 * b.tb);  // no new token of the block sees one before
      const int y = next_y, count = each * S::KT;
      const uint32_t copied = __ballot_sync(0xffffffffu, y >= 0);
      const bool whole = count == 8 * S::KT && copied == (uint32_t)((1ull << (8 * S::KT)) - 1);
      int ys[8 * S::KT];
#pragma unroll
      for (int k = 0; k < 8 * S::KT; ++k) ys[k] = __shfl_sync(0xffffffffu, y, k);
      bool first_unit = true;
      each_unit(sp, [&](uint32_t, int kvh, int piece, int i, bool first, bool) {
        if (first && warp == S::kLoad) {
          const uint32_t set = sets % S::SETS, parity = (sets / S::SETS & 1) ^ 1;
          const uint32_t to = sb + S::k + set * S::kSet;
          const int kcol = gqa ? kvh * lay.hd : 0;
          ++sets;
          if (whole) {  // a warp alone takes some five cycles an instruction: few of them
            if (ptx::elect_one()) {
#pragma unroll 1
              for (int c = 0; c < S::DK; ++c) {
                const uint32_t full = bar(S::k_full + set * S::DK + c);
                wait(bar(S::k_empty + set * S::DK + c), parity);
                if (dead) break;
                ptx::mbar_arrive_n(full, 31);
                ptx::mbar_arrive_expect_tx(full, S::KT * kChunk);
#pragma unroll
                for (int k = 0; k < 8 * S::KT; ++k)
                  ptx::tma_2d(to + c * S::KT * kChunk + k * 2048, &maps.k, kcol + c * 64, ys[k], full);
              }
            }
            __syncwarp();
          } else if (box) {
#pragma unroll 1
            for (int c = 0; c < S::DK; ++c) {
              const uint32_t full = bar(S::k_full + set * S::DK + c);
              wait(bar(S::k_empty + set * S::DK + c), parity);
              if (ptx::elect_one() && !dead) {
                ptx::mbar_arrive_n(full, 31);
                ptx::mbar_arrive_expect_tx(full, __popc(copied) * box * 128);
#pragma unroll
                for (int k = 0; k < 8 * S::KT; ++k)
                  if (copied >> k & 1)
                    ptx::tma_2d(to + c * S::KT * kChunk + k * box * 128, &maps.k, kcol + c * 64, ys[k],
                                full);
              }
              __syncwarp();
#pragma unroll 1
              for (int k = 8 * S::KT; k < count; ++k) {  // (pages of 8 slots)
                const int row = __shfl_sync(0xffffffffu, y, k);
                if (ptx::elect_one() && !dead && row >= 0)
                  ptx::tma_2d(to + c * S::KT * kChunk + k * box * 128, &maps.k, kcol + c * 64, row,
                              full);
              }
            }
          } else {
            const int p = lane & 7;  // 16-byte piece of a row
            const __nv_bfloat16 *base = b.pool.k +
                                        (long long)b.layer * b.pool.num_slots * lay.row_k + kcol + 8 * p;
            int slot[4 * S::KT];
#pragma unroll
            for (int k = 0; k < 4 * S::KT; ++k) {
              const long long tok = (long long)tok0 + 32 * k + lane;
              slot[k] = tok >= lo && tok < ctx ? slot_in(b, load_page(b, r, (int)tok), (int)tok) : -1;
            }
#pragma unroll 1
            for (int c = 0; c < S::DK; ++c) {
              wait(bar(S::k_empty + set * S::DK + c), parity);
              if (__any_sync(0xffffffffu, dead)) {
                dead = true;
                continue;
              }
#pragma unroll
              for (int k = 0; k < 4 * S::KT; ++k)
#pragma unroll 2
                for (int j = 0; j < 8; ++j) {  // four tokens at a time
                  const int row = 32 * k + 4 * j + (lane >> 3);
                  const int sl = __shfl_sync(0xffffffffu, slot[k], 4 * j + (lane >> 3));
                  ptx::cp_async16(to + c * S::KT * kChunk + row * 128 + ((p ^ (row & 7)) << 4),
                                  base + (long long)max(sl, 0) * lay.row_k + c * 64,
                                  sl >= 0 ? 16u : 0u);
                }
              ptx::cp_async_commit();
              ptx::cp_async_wait_all();
              ptx::fence_proxy_async_smem();
              ptx::mbar_arrive(bar(S::k_full + set * S::DK + c));
            }
          }
        }
        // Q. Rows of a copy past the tile's are other tokens' or zero: they are left out by their
        // log-sum-exps
        const int h0 = kvh * b.hpk + piece * a.shape.qr, z = sp->row + i * b.tb;
        const bool one = min(b.tb, sp->n - i * b.tb) == 1;
        const int bytes = one ? maps.token_bytes : maps.block_bytes;
        if (warp == S::kQ && ptx::elect_one()) {
#pragma unroll 1
          for (int s = 0; s < S::DK / S::UC; ++s) {
            const uint32_t n = stages + s, at = n % S::NST, full = bar(S::q_full) + 8 * at;
            wait(bar(S::q_empty) + 8 * at, (n / S::NST & 1) ^ 1);
            if (dead) break;
            ptx::mbar_arrive_expect_tx(full, bytes * S::UC);
#pragma unroll
            for (int c = 0; c < S::UC; ++c)
              ptx::tma_3d(sb + S::ring + at * S::kStage + c * kChunk,
                          one ? &maps.q_token : &maps.q_block, (s * S::UC + c) * 64, h0, z, full);
          }
        }
        __syncwarp();
        stages += S::DK / S::UC;
        if (first_unit) {
          publish();
          if (warp == S::kLoad) next_y = look_up(segs + (published - 1) % kSegs);
        }
        first_unit = false;
      });
    }
    ptx::cp_async_wait_all();
  } else if (warp == S::kLse) {
    // ---- c' lse of the query rows, four a lane, and how the weights are to be taken ----
    const float inf = __int_as_float(0x7f800000);
    float *z = reinterpret_cast<float *>(smem + S::z);
    const bool counts = b.scale != 0.f;
    while (const Seg *sp = take_whole()) {
      each_unit(sp, [&](uint32_t u, int kvh, int piece, int i, bool, bool) {
        const uint32_t zs = u % kZ;
        const int ntok = min(b.tb, sp->n - i * b.tb), h0 = kvh * b.hpk + piece * a.shape.qr;
        const int heads = min(b.hpk - piece * a.shape.qr, a.shape.qr), rows = ntok * heads;
        const float *lse = a.lse + (long long)(sp->row + i * b.tb) * b.hq + h0;
        float v[4];
        bool finite = counts;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int row = 32 * k + lane;
          const int d = b.pieces > 1 ? 0 : (int)((unsigned)row * b.hpk_magic >> 16);
          v[k] = row < rows ? lse[(long long)d * b.hq + row - d * b.hpk] : inf;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          finite = finite && (32 * k + lane >= rows || fabsf(v[k]) < inf);
          v[k] = v[k] == -inf ? inf : v[k] * kLog2e;  // what saw nothing lays nothing on any token
        }
        finite = __all_sync(0xffffffffu, finite);
        if (u >= kZ) wait(bar(S::z_free) + 8 * zs, (u / kZ & 1) ^ 1);
#pragma unroll
        for (int k = 0; k < 4; ++k) z[zs * kRow + 32 * k + lane] = v[k];
        if (lane == 0) {
          const int first = sp->past + i * b.tb;
          // (rows that a copy of a whole tile does not write are 0, others may be anything)
          const bool full = ntok == b.tb && heads == min(b.hpk, a.shape.qr);
          int how[2] = {0, 0};
#pragma unroll
          for (int w = 0; w < S::KT; ++w) {
            const int t0 = sp->tok0 + w * kTok;
            how[w] = !finite ? 2
                             : !(full && first + 1 - t0 >= kTok &&
                                 first_seen(b, first + ntok - 1) <= t0);
          }
          *reinterpret_cast<int4 *>(smem + S::flags + 16 * zs) =
              make_int4(rows, how[0], how[1], i * b.tb);
        }
        __syncwarp();
        if (lane == 0 && !dead) ptx::mbar_arrive(bar(S::z_full) + 8 * zs);
      });
    }
  } else if (warp < S::kMma + S::KT && ptx::elect_one()) {
    // ---- MMAs, one thread for each tile of tokens ----
    const int w = warp - S::kMma;
    constexpr uint32_t id =
        1u << 4 | 1u << 7 | 1u << 10 | (kRow >> 3) << 17 | (kTok >> 4) << 24;
    const uint32_t k0 = desc_k(sb + S::k) + w * (kChunk >> 4), q0 = desc_k(sb + S::ring);
    uint32_t sets = 0, stages = 0;
    while (const Seg *sp = take_segment()) {
      each_unit(sp, [&](uint32_t u, int, int, int, bool first, bool last) {
        const uint32_t set = sets % S::SETS;
        uint32_t n = u * S::kPieces, buf = 0;  // the next piece's number, the present one's buffer
#pragma unroll 1
        for (int s = 0; s < S::DK / S::UC; ++s, ++stages) {
          const uint32_t at = stages % S::NST;
          const bool begins_piece = s * S::UC % S::AC == 0;
          if (begins_piece) {
            buf = w * S::kBuf + n % S::kBuf;
            if (n >= S::kBuf) wait(bar(S::s_free) + 8 * buf, (n / S::kBuf & 1) ^ 1);
            if (!dead) ptx::tc_fence_after();
            ++n;
          }
          if (first)
            for (int c = 0; c < S::UC; ++c)
              wait(bar(S::k_full + set * S::DK + s * S::UC + c), sets / S::SETS & 1);
          wait(bar(S::q_full) + 8 * at, stages / S::NST & 1);
          if (dead) return;
          const uint32_t kd = k0 + ((set * S::kSet + s * S::UC * S::KT * kChunk) >> 4);
          const uint32_t qd = q0 + (at * S::kStage >> 4);
#pragma unroll
          for (int x = 0; x < S::UC * 4; ++x)
            ptx::mma_bf16(tmem + buf * 128,
                          desc(kd + (((x >> 2) * S::KT * kChunk + (x & 3) * 32) >> 4)),
                          desc(qd + (((x >> 2) * kChunk + (x & 3) * 32) >> 4)), id,
                          !begins_piece || x ? 1u : 0u);
          ptx::mma_commit(bar(S::q_empty) + 8 * at);
          if (last)
            for (int c = 0; c < S::UC; ++c)
              ptx::mma_commit(bar(S::k_empty + set * S::DK + s * S::UC + c));
          if ((s + 1) * S::UC % S::AC == 0 || (s + 1) * S::UC == S::DK)
            ptx::mma_commit(bar(S::s_full) + 8 * buf);
        }
        if (last) ++sets;
      });
    }
    ptx::mma_commit(bar(S::last + w));  // no MMA is in flight when the TMEM goes back
    if (!ptx::mbar_wait(bar(S::last + w), 0, kPrefixWaitNs)) *gave_up = 1;
  }
  __syncwarp();
  ptx::tc_fence_before();
  __syncthreads();
  if (tid == 0) places.rec[blockIdx.x].gave_up = *gave_up;
  if (*gave_up) {  // copies and MMAs in flight end long before this
    if (tid == 0) atomicOr(b.status, KAMERA_DEVICE_TIMEOUT);
    const uint64_t t0 = ptx::globaltimer();
    while (ptx::globaltimer() - t0 < 1000000) {
    }
    __syncthreads();
  }
  if (warp == S::kMma) ptx::tmem_dealloc(tmem, 512);
}

template <class S>
cudaError_t configure() {
  return cudaFuncSetAttribute(mass_tc_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              S::total);
}

template <class S>
cudaError_t launch(const MassArgs &a, cudaStream_t s) {
  if (!encode_fn()) return cudaErrorNotSupported;
  Maps m;
  const ChunkArgs &b = a.b;
  const DevLayout &l = b.lay;
  const int ps = l.page_size, heads = b.hpk < a.shape.qr ? b.hpk : a.shape.qr;
  m.box = ps % kTok == 0 ? kTok : (ps >= 8 && kTok % ps == 0 ? ps : 0);
  const uint32_t box = m.box ? m.box : 8;
  m.copies = kTok / box;
  m.per_page = ps >= kTok ? ps / kTok : 1;
  const __nv_bfloat16 *k = b.pool.k + b.layer * b.pool.num_slots * l.row_k;
  const bool ok =
      encode(&m.k, k, 2, l.row_k, b.pool.num_slots, 1, l.row_k, 0, box, 1) &&
      encode(&m.q_block, b.q, 3, b.dk, b.hq, b.n_tokens, b.dk, b.q_stride, heads, b.tb) &&
      encode(&m.q_token, b.q, 3, b.dk, b.hq, b.n_tokens, b.dk, b.q_stride, heads, 1);
  if (!ok) return cudaErrorInvalidValue;
  m.token_bytes = 128 * heads;
  m.block_bytes = m.token_bytes * b.tb;
  mass_tc_kernel<S><<<a.shape.n, S::kThr, S::total, s>>>(a, m);
  return cudaGetLastError();
}

}  // namespace

MassShape mass_tc_shape(const DevLayout &l) {
  return {l.kind == KAMERA_MLA ? kTok : 2 * kTok, kRow, kSms};
}

cudaError_t prepare_mass_tc(const DevLayout &l) {
  if (l.kind == KAMERA_MLA) return configure<Mla512>();
  return l.hd == 128 ? configure<Gqa128>() : configure<Gqa64>();
}

cudaError_t launch_mass_tc(const MassArgs &a, cudaStream_t s) {
  if (a.b.lay.kind == KAMERA_MLA) return launch<Mla512>(a, s);
  return a.b.lay.hd == 128 ? launch<Gqa128>(a, s) : launch<Gqa64>(a, s);
}

}  // namespace kamera
