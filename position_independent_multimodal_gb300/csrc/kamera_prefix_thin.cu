// Thin blocks of attention over shared prefixes: at most 16 query rows against long rows of
// tokens, as one request's heads of a KV head are. The bytes of K and V bound them, so the work is
// laid out for loads: m16n8k16 tensor-core products on registers (16 rows are one such tile; a
// tcgen05 tile would have 128), K and V straight from the page rows by cp.async, several stages
// ahead and across the ends of segments.
//
//   S = Q K^T, P = bf16(2^(c S - m)), O += P V,  c = scale log2 e,  m raised by at least 8 at once
//
// Sums l and maxima m are float32 and l takes the unrounded weights. P is rounded to bf16, as the
// products with bf16 V want it; the reasons and the error are with the wide blocks' kernel, and
// rows that both kernels work on have one accuracy.
//
//  * prefix_thin_kernel (GQA, head_dim 64 or 128): each warp is a worker with a range of 16-token
//    tiles of its own and its own ring of stages (K, V and, with a segment's first tile, Q); the
//    warps of a CTA share nothing, so nothing waits for another warp. 128 requests' own tokens
//    (500 at most) of 28/4 heads of 128: 22 us, 66 MB read, 3 TB/s. The start and each warp's chain
//    of a tile's products and softmax bound it; eleven warps of two stages are slower than these
//    six of three.
//  * prefix_thin_mla_kernel (latent 512 + 64): a row of K is 1152 bytes and O has 512 columns, so
//    eight warps work on one tile of 64 tokens: eight tokens of S each, then 64 columns of O each.
//    40 requests' own tokens (300 at most): 9 to 11 us, the start for the most part.
#include "kamera_prefix.cuh"
#include "kamera_ptx.cuh"

namespace kamera {

namespace {

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t *r) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
// D [16 x 8] += A [16 x 16] B [16 x 8], bf16 in, float32 out
__device__ __forceinline__ void mma16816(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr int kRows = 16;

// ---------------------------------------------------------------------------------------
// GQA
// ---------------------------------------------------------------------------------------

template <int D_, int WARPS_, int NST_>
struct Thin {
  static constexpr int D = D_, WARPS = WARPS_, NST = NST_;
  static constexpr int kTok = 16;
  static constexpr int kTile = kTok * D * 2;    // bytes of a tile of K, of V and of Q
  static constexpr int kStage = 3 * kTile;
  static constexpr int queue = WARPS * NST * kStage;  // Segment [WARPS][8]
  static constexpr int total = queue + WARPS * 8 * (int)sizeof(Segment);
  static constexpr int pieces = D / 8;          // 16-byte pieces of a row
  static_assert(NST <= 4, "token masks of the stages share a 64-bit register");
};
using Thin128 = Thin<128, 6, 3>;
using Thin64 = Thin<64, 8, 4>;

// Byte offset of a 16-byte piece of a row: eight rows' pieces fall on distinct banks.
template <int D>
__device__ __forceinline__ uint32_t at16(int row, int piece) {
  if (D == 64) return row * 128 + ((piece ^ (row & 7)) << 4);
  return row * 256 + ((piece ^ (row & 7)) << 4);
}

template <class T>
__global__ void __launch_bounds__(T::WARPS * 32, 1)
    prefix_thin_kernel(const __grid_constant__ PrefixArgs a, int beside) {
  extern __shared__ __align__(128) unsigned char smem[];
  constexpr int D = T::D, kTok = T::kTok;
  const PrefixPlan plan = prefix_plan(a.shape, a.ws, a.n_reqs, a.hq, a.dv);
  const DevLayout &lay = a.lay;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int worker = warp * kSms + blockIdx.x;  // few units: one warp on each SM first
  const uint32_t ring = ptx::smem_addr(smem) + warp * (T::NST * T::kStage);
  const __nv_bfloat16 *lk = a.pool.k + (long long)a.layer * a.pool.num_slots * lay.row_k;
  const __nv_bfloat16 *lv = a.pool.v + (long long)a.layer * a.pool.num_slots * lay.row_v;
  const float neg_inf = -__int_as_float(0x7f800000);
  const float c = a.scale * kLog2e;

  // `beside`: the kernel before this one is that of the wide blocks, else the plan
  if (!beside) ptx::wait_for_previous();
  ptx::launch_dependents();

  // ---- loads: one tile ahead of its issue the page entry, NST - 1 tiles ahead of its use. The
  // segments go on through a queue: at most NST + 1 are between the loads and the products ----
  Segment *queue = reinterpret_cast<Segment *>(smem + T::queue) + warp * 8;
  SegmentWalk<1> lw;
  lw.start(a, plan, worker);
  Segment ls;
  int l_seg = 0;
  auto next_segment = [&]() {
    if (!lw.next(a, plan, &ls)) ls.rows = 0;  // the end
    if (lane == 0) queue[l_seg & 7] = ls;
    ++l_seg;
    return ls.rows > 0;
  };
  bool l_any = next_segment(), l_first = true;
  int l_t = l_any ? ls.tok0 / kTok : 0;  // tile to issue next
  int page = 0;                          // of lane's token of that tile
  auto fetch = [&]() {
    const int tok = l_t * kTok + (lane & 15);
    page = l_any && tok >= ls.tok0 && tok < ls.tok1 ? load_page(a, ls.lead, tok) : 0;
  };
  fetch();
  uint64_t masks = 0;  // 16 bits for each stage
  int l_st = 0;        // stage to fill
  auto issue = [&]() {
    if (l_any) {
      const int tok = l_t * kTok + (lane & 15);
      const int slot = tok >= ls.tok0 && tok < ls.tok1 ? slot_in(a, page, tok) : -1;
      const uint32_t bits = __ballot_sync(0xffffffffu, slot >= 0) & 0xffffu;
      masks = (masks & ~(0xffffull << (16 * l_st))) | (uint64_t)bits << (16 * l_st);
      const uint32_t dst = ring + l_st * T::kStage;
      constexpr int step = 32 / T::pieces;  // rows a warp copies at once
      const int piece = lane % T::pieces, r0 = lane / T::pieces;
      const __nv_bfloat16 *kb = lk + ls.kvh * D + 8 * piece, *vb = lv + ls.kvh * D + 8 * piece;
#pragma unroll
      for (int j = 0; j < kTok / step; ++j) {
        const int r = r0 + j * step;
        const int sl = __shfl_sync(0xffffffffu, slot, r);
        const uint32_t d = dst + at16<D>(r, piece), n = sl >= 0 ? 16u : 0u;
        ptx::cp_async16(d, sl >= 0 ? kb + (long long)sl * lay.row_k : lk, n);
        ptx::cp_async16(d + T::kTile, sl >= 0 ? vb + (long long)sl * lay.row_v : lv, n);
      }
      if (l_first) {  // the segment's queries; rows that the block does not have are zero
#pragma unroll
        for (int j = 0; j < kRows / step; ++j) {
          const int i = r0 + j * step;
          const __nv_bfloat16 *src = a.q;
          if (i < ls.rows) {
            int r, h;
            segment_row(a, ls, i, &r, &h);
            src += ((long long)r * a.hq + h) * D + 8 * piece;
          }
          ptx::cp_async16(dst + 2 * T::kTile + at16<D>(i, piece), src, i < ls.rows ? 16u : 0u);
        }
      }
      l_first = false;
      if (++l_t >= ceil_div(ls.tok1, kTok)) {
        l_any = next_segment();
        l_first = true;
        if (l_any) l_t = ls.tok0 / kTok;
      }
      fetch();
    }
    ptx::cp_async_commit();
    l_st = l_st + 1 == T::NST ? 0 : l_st + 1;
  };
  // a loop: code is fetched cold by every SM, and a copy for each stage costs 6 us a call
#pragma unroll 1
  for (int i = 0; i < T::NST - 1; ++i) issue();

  // ---- attention ----
  int st = 0;
  const int g = lane >> 2, q4 = lane & 3;  // rows g and g + 8, columns 2 q4, 2 q4 + 1
  for (int seg = 0;; ++seg) {
    __syncwarp();
    const Segment s = queue[seg & 7];
    if (s.rows == 0) break;
    uint32_t qf[D / 16][4];
    float o[D / 8][4], m0 = neg_inf, m1 = neg_inf, l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int j = 0; j < D / 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    const int ta = s.tok0 / kTok, tb = ceil_div(s.tok1, kTok);
    for (int t = ta; t < tb; ++t) {
      cp_wait<T::NST - 2>();
      __syncwarp();  // the tile has landed for every lane; the stage before it has been read
      const uint32_t bits = (uint32_t)(masks >> (16 * st)) & 0xffffu;
      issue();
      const uint32_t kb = ring + st * T::kStage, vb = kb + T::kTile;
      if (t == ta) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          ldsm4(kb + 2 * T::kTile + at16<D>(lane & 15, 2 * k + (lane >> 4)), qf[k]);
      }
      float x[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
      for (int k = 0; k < D / 16; ++k) {  // tokens 0-7 and 8-15, 16 dims
        uint32_t b[4];
        ldsm4(kb + at16<D>((lane & 7) + ((lane >> 4) << 3), 2 * k + ((lane >> 3) & 1)), b);
        mma16816(x[0], qf[k], b[0], b[1]);
        mma16816(x[1], qf[k], b[2], b[3]);
      }
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[j][e] *= c;
      if (bits != 0xffffu) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (!((bits >> (8 * j + 2 * q4 + (e & 1))) & 1)) x[j][e] = neg_inf;
      }
      float t0 = fmaxf(fmaxf(x[0][0], x[0][1]), fmaxf(x[1][0], x[1][1]));
      float t1 = fmaxf(fmaxf(x[0][2], x[0][3]), fmaxf(x[1][2], x[1][3]));
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
      }
      // raised from -inf (nothing seen) or by more than a factor 2^8 in P
      const bool up0 = t0 > m0 + 8.f, up1 = t1 > m1 + 8.f;
      if (__any_sync(0xffffffffu, up0 || up1)) {
        const float f0 = up0 ? exp2_approx(m0 - t0) : 1.f, f1 = up1 ? exp2_approx(m1 - t1) : 1.f;
        if (up0) m0 = t0;
        if (up1) m1 = t1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int j = 0; j < D / 8; ++j) {
          o[j][0] *= f0;
          o[j][1] *= f0;
          o[j][2] *= f1;
          o[j][3] *= f1;
        }
      }
      const float b0 = m0 > neg_inf ? m0 : 0.f, b1 = m1 > neg_inf ? m1 : 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        x[j][0] = exp2_approx(x[j][0] - b0);
        x[j][1] = exp2_approx(x[j][1] - b0);
        x[j][2] = exp2_approx(x[j][2] - b1);
        x[j][3] = exp2_approx(x[j][3] - b1);
        l0 += x[j][0] + x[j][1];
        l1 += x[j][2] + x[j][3];
      }
      const uint32_t p[4] = {pack_bf16(x[0][0], x[0][1]), pack_bf16(x[0][2], x[0][3]),
                             pack_bf16(x[1][0], x[1][1]), pack_bf16(x[1][2], x[1][3])};
#pragma unroll
      for (int j = 0; j < D / 16; ++j) {  // 16 columns of V
        uint32_t b[4];
        ldsm4t(vb + at16<D>(lane & 15, 2 * j + (lane >> 4)), b);
        mma16816(o[2 * j], p, b[0], b[1]);
        mma16816(o[2 * j + 1], p, b[2], b[3]);
      }
      st = st + 1 == T::NST ? 0 : st + 1;
    }
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = g + 8 * half;
      if (i >= s.rows) continue;
      const float l = half ? l1 : l0, m = half ? m1 : m0;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float *dst, *lse;
      segment_out<1>(a, plan, s, worker, i, q4 == 0, &dst, &lse);
#pragma unroll
      for (int j = 0; j < D / 8; ++j) {
        const float2 v = make_float2(l == 0.f ? 0.f : o[j][2 * half] * inv,
                                     l == 0.f ? 0.f : o[j][2 * half + 1] * inv);
        *reinterpret_cast<float2 *>(dst + 8 * j + 2 * q4) = v;
      }
      if (q4 == 0) *lse = l == 0.f ? neg_inf : (m + log2f(l)) * kLn2;
    }
  }
  cp_wait<0>();
  if (beside) ptx::wait_for_previous();  // who waits for this kernel waits for that one too
}

// ---------------------------------------------------------------------------------------
// MLA, latent 512 + 64
// ---------------------------------------------------------------------------------------

struct ThinMla {
  static constexpr int D = 576, kTok = 64, kThr = 256;
  static constexpr int kRow = D * 2;            // bytes of a row
  static constexpr int kTile = kTok * kRow;
  static constexpr int k = 0;                   // two stages
  static constexpr int q = 2 * kTile;           // two blocks' queries
  static constexpr int p = q + 2 * kRows * kRow;     // P [16][64] bf16
  static constexpr int slot = p + kRows * kTok * 2;  // int [4][kTok]
  static constexpr int wmax = slot + 4 * kTok * 4;   // float [8][16]
  static constexpr int wsum = wmax + 8 * kRows * 4;  // float [8][16]
  static constexpr int queue = wsum + 8 * kRows * 4;  // Segment [8]
  static constexpr int total = queue + 8 * (int)sizeof(Segment);
};

// Byte offset of a 16-byte piece (0..71) of a row.
__device__ __forceinline__ uint32_t mla16(int row, int piece) {
  return row * ThinMla::kRow + ((piece ^ (row & 7)) << 4);
}

__global__ void __launch_bounds__(ThinMla::kThr, 1)
    prefix_thin_mla_kernel(const __grid_constant__ PrefixArgs a, int beside) {
  extern __shared__ __align__(128) unsigned char smem[];
  using M = ThinMla;
  const PrefixPlan plan = prefix_plan(a.shape, a.ws, a.n_reqs, a.hq, a.dv);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, q4 = lane & 3;
  const uint32_t sb = ptx::smem_addr(smem);
  const __nv_bfloat16 *lk = a.pool.k + (long long)a.layer * a.pool.num_slots * M::D;
  int *slots = reinterpret_cast<int *>(smem + M::slot);
  float *wmax = reinterpret_cast<float *>(smem + M::wmax);
  float *wsum = reinterpret_cast<float *>(smem + M::wsum);
  const float neg_inf = -__int_as_float(0x7f800000);
  const float c = a.scale * kLog2e;

  if (!beside) ptx::wait_for_previous();
  ptx::launch_dependents();

  // ---- loads: slots two tiles ahead, rows one tile ahead ----
  Segment *queue = reinterpret_cast<Segment *>(smem + M::queue);
  SegmentWalk<1> sw;  // of the slots; the segments go on through the queue
  sw.start(a, plan, blockIdx.x);
  Segment ss;
  int s_seg = 0;
  auto next_segment = [&]() {
    if (!sw.next(a, plan, &ss)) ss.rows = 0;  // the end
    if (tid == 0) queue[s_seg & 7] = ss;
    ++s_seg;
    return ss.rows > 0;
  };
  bool s_any = next_segment();
  int s_t = s_any ? ss.tok0 / M::kTok : 0, s_no = 0;
  auto resolve = [&]() {  // the next tile's slots, one thread a token
    if (!s_any) return;
    if (tid < M::kTok) {
      const int tok = s_t * M::kTok + tid;
      slots[(s_no & 3) * M::kTok + tid] =
          tok >= ss.tok0 && tok < ss.tok1 ? slot_in(a, load_page(a, ss.lead, tok), tok) : -1;
    }
    ++s_no;
    if (++s_t >= ceil_div(ss.tok1, M::kTok)) {
      s_any = next_segment();
      if (s_any) s_t = ss.tok0 / M::kTok;
    }
  };
  Segment ls;
  bool l_any = true, l_first = true;
  int l_t = 0, l_no = 0, l_seg = 0;
  auto load_segment = [&]() {
    ls = queue[l_seg & 7];
    l_any = ls.rows > 0;
    l_first = true;
    l_t = ls.tok0 / M::kTok;
  };
  auto issue = [&]() {  // rows of the next tile, whose slots are there
    if (l_any) {
      const uint32_t dst = sb + M::k + (l_no & 1) * M::kTile;
      const int *sl = slots + (l_no & 3) * M::kTok;
      // 72 pieces a row: eight threads take a 128-byte line of it at a time
      const int x = tid & 7, y = tid >> 3;
#pragma unroll
      for (int j = 0; j < M::kTok / 32; ++j) {
        const int r = y + 32 * j, s = sl[r];
        const __nv_bfloat16 *src = s >= 0 ? lk + (long long)s * M::D + 8 * x : lk;
#pragma unroll
        for (int k = 0; k < 9; ++k)
          ptx::cp_async16(dst + mla16(r, x + 8 * k), s >= 0 ? src + 64 * k : src,
                          s >= 0 ? 16u : 0u);
      }
      if (l_first) {
        const int i = y;  // 16 rows, by half of the threads
        if (i < kRows) {
          const __nv_bfloat16 *src = a.q;
          if (i < ls.rows) {
            int r, h;
            segment_row(a, ls, i, &r, &h);
            src += ((long long)r * a.hq + h) * M::D + 8 * x;
          }
#pragma unroll
          for (int k = 0; k < 9; ++k)
            ptx::cp_async16(sb + M::q + (l_seg & 1) * (kRows * M::kRow) + mla16(i, x + 8 * k),
                            i < ls.rows ? src + 64 * k : src, i < ls.rows ? 16u : 0u);
        }
      }
      l_first = false;
      ++l_no;
      if (++l_t >= ceil_div(ls.tok1, M::kTok)) {
        ++l_seg;
        load_segment();
      }
    }
    ptx::cp_async_commit();
  };
  resolve();
  resolve();
  __syncthreads();
  load_segment();
  issue();

  int no = 0;
  for (int seg = 0;; ++seg) {
    const Segment s = queue[seg & 7];
    if (s.rows == 0) break;
    float o[8][4], m0 = neg_inf, m1 = neg_inf, l0 = 0.f, l1 = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j][0] = o[j][1] = o[j][2] = o[j][3] = 0.f;
    const uint32_t qb = sb + M::q + (seg & 1) * (kRows * M::kRow);
    const int ta = s.tok0 / M::kTok, tb = ceil_div(s.tok1, M::kTok);
    for (int t = ta; t < tb; ++t, ++no) {
      cp_wait<0>();
      __syncthreads();  // the tile has landed; the other stage, P and the statistics are free
      issue();
      resolve();
      const uint32_t kb = sb + M::k + (no & 1) * M::kTile;
      const int *sl = slots + (no & 3) * M::kTok + 8 * warp + 2 * q4;
      const bool in0 = sl[0] >= 0, in1 = sl[1] >= 0;
      float x[4] = {0.f, 0.f, 0.f, 0.f}, y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 6
      for (int k = 0; k < M::D / 32; ++k) {  // eight tokens of this warp, 32 dims
        uint32_t b[4], q0[4], q1[4];
        ldsm4(kb + mla16(8 * warp + (lane & 7), 4 * k + (lane >> 3)), b);
        ldsm4(qb + mla16(lane & 15, 4 * k + (lane >> 4)), q0);
        ldsm4(qb + mla16(lane & 15, 4 * k + 2 + (lane >> 4)), q1);
        mma16816(x, q0, b[0], b[1]);
        mma16816(y, q1, b[2], b[3]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = (x[e] + y[e]) * c;
      if (!in0) x[0] = x[2] = neg_inf;
      if (!in1) x[1] = x[3] = neg_inf;
      float t0 = fmaxf(x[0], x[1]), t1 = fmaxf(x[2], x[3]);
#pragma unroll
      for (int d = 1; d < 4; d <<= 1) {
        t0 = fmaxf(t0, __shfl_xor_sync(0xffffffffu, t0, d));
        t1 = fmaxf(t1, __shfl_xor_sync(0xffffffffu, t1, d));
      }
      if (q4 == 0) {
        wmax[warp * kRows + g] = t0;
        wmax[warp * kRows + g + 8] = t1;
      }
      __syncthreads();
#pragma unroll
      for (int w = 0; w < 8; ++w) {
        t0 = fmaxf(t0, wmax[w * kRows + g]);
        t1 = fmaxf(t1, wmax[w * kRows + g + 8]);
      }
      const bool up0 = t0 > m0 + 8.f, up1 = t1 > m1 + 8.f;  // alike in every warp
      if (__any_sync(0xffffffffu, up0 || up1)) {
        const float f0 = up0 ? exp2_approx(m0 - t0) : 1.f, f1 = up1 ? exp2_approx(m1 - t1) : 1.f;
        if (up0) m0 = t0;
        if (up1) m1 = t1;
        l0 *= f0;
        l1 *= f1;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          o[j][0] *= f0;
          o[j][1] *= f0;
          o[j][2] *= f1;
          o[j][3] *= f1;
        }
      }
      const float b0 = m0 > neg_inf ? m0 : 0.f, b1 = m1 > neg_inf ? m1 : 0.f;
      x[0] = exp2_approx(x[0] - b0);
      x[1] = exp2_approx(x[1] - b0);
      x[2] = exp2_approx(x[2] - b1);
      x[3] = exp2_approx(x[3] - b1);
      l0 += x[0] + x[1];
      l1 += x[2] + x[3];
      // P [16][64]: rows of 128 bytes, pieces swizzled as the operands'
      unsigned char *pp = smem + M::p;
      *reinterpret_cast<uint32_t *>(pp + g * 128 + ((warp ^ (g & 7)) << 4) + 4 * q4) =
          pack_bf16(x[0], x[1]);
      *reinterpret_cast<uint32_t *>(pp + (g + 8) * 128 + ((warp ^ (g & 7)) << 4) + 4 * q4) =
          pack_bf16(x[2], x[3]);
      __syncthreads();
#pragma unroll
      for (int k = 0; k < M::kTok / 16; ++k) {  // 16 tokens, this warp's 64 columns
        uint32_t pa[4];
        const int r = lane & 15;
        ldsm4(sb + M::p + r * 128 + (((2 * k + (lane >> 4)) ^ (r & 7)) << 4), pa);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t b[4];
          ldsm4t(kb + mla16(16 * k + (lane & 15), 8 * warp + 2 * j + (lane >> 4)), b);
          mma16816(o[2 * j], pa, b[0], b[1]);
          mma16816(o[2 * j + 1], pa, b[2], b[3]);
        }
      }
    }
    // sums over the warps' tokens
#pragma unroll
    for (int d = 1; d < 4; d <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, d);
      l1 += __shfl_xor_sync(0xffffffffu, l1, d);
    }
    if (q4 == 0) {
      wsum[warp * kRows + g] = l0;
      wsum[warp * kRows + g + 8] = l1;
    }
    __syncthreads();
    l0 = l1 = 0.f;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      l0 += wsum[w * kRows + g];
      l1 += wsum[w * kRows + g + 8];
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const int i = g + 8 * half;
      if (i >= s.rows) continue;
      const float l = half ? l1 : l0, m = half ? m1 : m0;
      const float inv = l == 0.f ? 0.f : 1.f / l;
      float *dst, *lse;
      segment_out<1>(a, plan, s, blockIdx.x, i, q4 == 0 && warp == 0, &dst, &lse);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 v = make_float2(l == 0.f ? 0.f : o[j][2 * half] * inv,
                                     l == 0.f ? 0.f : o[j][2 * half + 1] * inv);
        *reinterpret_cast<float2 *>(dst + 64 * warp + 8 * j + 2 * q4) = v;
      }
      if (q4 == 0 && warp == 0) *lse = l == 0.f ? neg_inf : (m + log2f(l)) * kLn2;
    }
  }
  cp_wait<0>();
  if (beside) ptx::wait_for_previous();
}

}  // namespace

PrefixClass prefix_thin_class(const DevLayout &l) {
  PrefixClass c;
  c.rb = kRows;
  c.vh = 1;
  if (l.kind == KAMERA_MLA) {
    c.tile_sh = 6;
    static_assert(ThinMla::kTok == 1 << 6, "a tile");
    c.n = kSms;
    c.least = 1;
  } else {
    c.tile_sh = 4;
    c.n = kSms * (l.hd == 128 ? Thin128::WARPS : Thin64::WARPS);
    c.least = 4;
  }
  return c;
}

cudaError_t prepare_prefix_thin(const DevLayout &l) {
  auto set = [](const void *f, int bytes) {
    return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  };
  if (l.kind == KAMERA_MLA) return set((const void *)prefix_thin_mla_kernel, ThinMla::total);
  if (l.hd == 128) return set((const void *)prefix_thin_kernel<Thin128>, Thin128::total);
  return set((const void *)prefix_thin_kernel<Thin64>, Thin64::total);
}

cudaError_t launch_prefix_thin(const PrefixArgs &a, bool beside, cudaStream_t s) {
  const int b = beside;
  if (a.lay.kind == KAMERA_MLA)
    return launch_early(prefix_thin_mla_kernel, dim3(kSms), ThinMla::kThr, ThinMla::total, s, a, b);
  if (a.lay.hd == 128)
    return launch_early(prefix_thin_kernel<Thin128>, dim3(kSms), Thin128::WARPS * 32,
                        Thin128::total, s, a, b);
  return launch_early(prefix_thin_kernel<Thin64>, dim3(kSms), Thin64::WARPS * 32, Thin64::total, s,
                      a, b);
}

}  // namespace kamera
