// Attention of chunks of new tokens over the paged pool: the kernel of the layouts that the
// tcgen05 kernel (kamera_chunk_tc.cu) does not take, and the join of the blocks that workers cut.
//
//   S = Q K^T,  P = 2^(c S - m),  O += P V,  l += sum P,  c = scale log2 e,  m the running maximum
//
// chunk_gen_kernel: m16n8k16 products on registers, four warps of 16 query rows, tiles of 32 tokens,
// at most 128 of V's columns a worker (wider V in parts, each with its own S). Widths are any
// multiple of 16, up to 1024. Bound by the loads of operands from shared memory, each used for one
// product: 54 TFLOP/s over 4 requests of 500 tokens over 4000 (16 query heads, 4 KV heads of 96), a
// batch of 32 that decode over 4000 in 285 us. Sums and maxima are float32; P is rounded to bf16 for
// the product with V, as in the other kernels of this kind, and l takes the unrounded weights.
#include <algorithm>
#include <mutex>

#include "kamera_chunk.cuh"
#include "kamera_mma.cuh"
#include "kamera_ptx.cuh"

namespace kamera {

namespace {

constexpr int kRows = 64, kTileSh = 5, kTile = 1 << kTileSh, kThr = 128, kCols = 128;

// Byte offsets of the shared memory.
struct GenPlan {
  int pitch, vpitch;  // of rows of Q and K, of V
  int q, k, v, total;
};
__host__ __device__ inline GenPlan gen_plan(int dk) {
  GenPlan p;
  p.pitch = 2 * dk + 16;
  p.vpitch = 2 * kCols + 16;
  p.q = 0;
  p.k = kRows * p.pitch;
  p.v = p.k + kTile * p.pitch;
  p.total = p.v + kTile * p.vpitch;
  return p;
}

__global__ void __launch_bounds__(kThr) chunk_gen_kernel(const __grid_constant__ ChunkArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ ChunkScratch<kThr> found;
  __shared__ uint32_t valid;  // tokens of the tile that have a slot
  __shared__ int slots[kTile];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, w = blockIdx.x;
  const DevLayout &lay = a.lay;
  const GenPlan pl = gen_plan(a.dk);
  const uint32_t sb = ptx::smem_addr(smem);
  const ChunkPlaces places = chunk_places(a.shape, a.ws);
  const bool gqa = lay.kind == KAMERA_GQA;
  const long long layer0 = (long long)a.layer * a.pool.num_slots;
  const __nv_bfloat16 *pk = a.pool.k + layer0 * lay.row_k;
  const __nv_bfloat16 *pv = gqa ? a.pool.v + layer0 * lay.row_v : pk;
  const int vrow = gqa ? lay.row_v : lay.row_k;
  const float neg_inf = -__int_as_float(0x7f800000);
  const float c = a.scale * kLog2e;
  const ChunkStart st = chunk_start<kThr>(a, w, &found);
  ptx::launch_dependents();
  ChunkWalk walk;
  walk.start(a, st, w);
  ChunkSegment s = {};
  int segments = 0;
  bool odd = false;  // an output is not finite
  for (; walk.next(a, &s); ++segments) {
    const int rows = s.ntok * s.heads;
    const int kcol = gqa ? s.kvh * lay.hd : 0, vcol = kcol + s.part * kCols;
    const int cols = min(kCols, a.dv - s.part * kCols);
    __syncthreads();
    const int qp = a.dk >> 3;  // 16-byte pieces of a row
    for (int e = tid; e < kRows * qp; e += kThr) {
      const int i = e / qp, p = e - i * qp;
      int k, h;
      chunk_row(a, s, i < rows ? i : 0, &k, &h);
      const __nv_bfloat16 *src = a.q + (s.row + k) * a.q_stride + (long long)h * a.dk + 8 * p;
      ptx::cp_async16(sb + pl.q + i * pl.pitch + 16 * p, src, i < rows ? 16u : 0u);
    }
    ptx::cp_async_commit();
    // what this thread's two rows see
    int see0[2], see1[2];
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      const int i = 16 * warp + 8 * y + (lane >> 2);
      int k, h;
      chunk_row(a, s, i < rows ? i : 0, &k, &h);
      see1[y] = s.first + k + 1;
      see0[y] = first_seen(a, s.first + k);
    }
    const int lo = first_seen(a, s.first);  // first token that a row sees
    float m[2] = {neg_inf, neg_inf}, l[2] = {0.f, 0.f};
    float o[kCols / 8][4];
#pragma unroll
    for (int n = 0; n < kCols / 8; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
    for (int t = s.t0; t < s.t1; ++t) {
      const int tok0 = t << kTileSh;
      __syncthreads();  // the tile before has been read
      if (tid < kTile) {
        const int tok = tok0 + tid;
        const int slot = tok >= lo && tok < s.ctx ? slot_in(a, load_page(a, s.r, tok), tok) : -1;
        slots[tid] = slot;
        const uint32_t in = __ballot_sync(0xffffffffu, slot >= 0);
        if (tid == 0) valid = in;
      }
      __syncthreads();
      for (int e = tid; e < kTile * qp; e += kThr) {
        const int i = e / qp, p = e - i * qp, slot = slots[i];
        ptx::cp_async16(sb + pl.k + i * pl.pitch + 16 * p,
                        slot >= 0 ? pk + (long long)slot * lay.row_k + kcol + 8 * p : pk,
                        slot >= 0 ? 16u : 0u);
      }
      const int vp = cols >> 3;
      for (int e = tid; e < kTile * vp; e += kThr) {
        const int i = e / vp, p = e - i * vp, slot = slots[i];
        ptx::cp_async16(sb + pl.v + i * pl.vpitch + 16 * p,
                        slot >= 0 ? pv + (long long)slot * vrow + vcol + 8 * p : pv,
                        slot >= 0 ? 16u : 0u);
      }
      ptx::cp_async_commit();
      ptx::cp_async_wait_all();
      __syncthreads();
      float x[kTile / 8][4];
#pragma unroll
      for (int n = 0; n < kTile / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
      for (int k = 0; k < a.dk; k += 16) {
        uint32_t qa[4];
        ldsm4(sb + pl.q + (16 * warp + (lane & 15)) * pl.pitch + 2 * k + 16 * (lane >> 4), qa);
#pragma unroll
        for (int n = 0; n < kTile / 16; ++n) {
          uint32_t kb[4];
          ldsm4(sb + pl.k + (16 * n + (lane & 7) + ((lane >> 4) << 3)) * pl.pitch + 2 * k +
                    16 * ((lane >> 3) & 1), kb);
          mma16816(x[2 * n], qa, kb[0], kb[1]);
          mma16816(x[2 * n + 1], qa, kb[2], kb[3]);
        }
      }
      const uint32_t in = valid;
      uint32_t pa[kTile / 16][4];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        float top = neg_inf;
#pragma unroll
        for (int n = 0; n < kTile / 8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = 8 * n + 2 * (lane & 3) + e;
            const bool on = ((in >> j) & 1) && tok0 + j >= see0[y] && tok0 + j < see1[y];
            float &v = x[n][2 * y + e];
            v = on ? v * c : neg_inf;
            top = fmaxf(top, v);
          }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const float next = fmaxf(m[y], top);
        const float base = next == neg_inf ? 0.f : next;
        const float f = m[y] == neg_inf ? 0.f : exp2_approx(m[y] - base);
        m[y] = next;
        float sum = 0.f;
#pragma unroll
        for (int n = 0; n < kTile / 8; ++n) {
          const float p0 = exp2_approx(x[n][2 * y] - base), p1 = exp2_approx(x[n][2 * y + 1] - base);
          sum += p0 + p1;
          pa[n >> 1][(n & 1) * 2 + y] = pack_bf16(p0, p1);
        }
        l[y] = l[y] * f + sum;
#pragma unroll
        for (int n = 0; n < kCols / 8; ++n) {
          o[n][2 * y] *= f;
          o[n][2 * y + 1] *= f;
        }
      }
#pragma unroll
      for (int k = 0; k < kTile / 16; ++k)
#pragma unroll
        for (int n = 0; n < kCols / 16; ++n) {
          if (16 * n >= cols) break;
          uint32_t vb[4];
          ldsm4t(sb + pl.v + (16 * k + (lane & 15)) * pl.vpitch + 32 * n + 16 * (lane >> 4), vb);
          mma16816(o[2 * n], pa[k], vb[0], vb[1]);
          mma16816(o[2 * n + 1], pa[k], vb[2], vb[3]);
        }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      l[y] += __shfl_xor_sync(0xffffffffu, l[y], 1);
      l[y] += __shfl_xor_sync(0xffffffffu, l[y], 2);
      const int i = 16 * warp + 8 * y + (lane >> 2);
      if (i >= rows) continue;
      int k, h;
      chunk_row(a, s, i, &k, &h);
      const float inv = l[y] == 0.f ? 0.f : 1.f / l[y];
      const float z = l[y] == 0.f ? neg_inf : (m[y] + log2f(l[y])) * kLn2;
      const long long rh = (long long)(s.row + k) * a.hq + h;
      const long long place = (long long)(2 * w + (s.carry() ? 0 : 1)) * kRows + i;
      const bool whole = chunk_whole(s);
#pragma unroll
      for (int n = 0; n < kCols / 8; ++n) {
        if (8 * n >= cols) break;
        const int col = 8 * n + 2 * (lane & 3);
        const float v0 = o[n][2 * y] * inv, v1 = o[n][2 * y + 1] * inv;
        odd |= v0 * 0.f + v1 * 0.f != 0.f;  // not finite
        if (whole)
          *reinterpret_cast<uint32_t *>(a.out + rh * a.dv + s.part * kCols + col) = pack_bf16(v0, v1);
        else
          *reinterpret_cast<float2 *>(places.o + place * kCols + col) = make_float2(v0, v1);
      }
      if ((lane & 3) == 0) {
        if (!whole)
          places.lse[place] = z;
        else if (s.part == 0)
          a.lse[rh] = z;
      }
    }
  }
  odd = __syncthreads_or(odd);
  if (tid == 0) chunk_note(places.rec + w, s, segments, false, odd);
}

// ---------------------------------------------------------------------------------------
// join
// ---------------------------------------------------------------------------------------

constexpr int kJoinThr = 256;

// One row of a block from its definition, token by token, by a warp: nothing that the row does not
// see is read. For blocks with values of V that are not finite in such places, which are rare: it is as
// slow as it is short. One such value among the last new tokens of 2011 over 60000 takes the call from 1.4
// to 380 ms, of 4 x 300 over 9003 (MLA) from 0.43 to 195, of a batch over 8000 from 0.35 to 44, with 64-wide
// heads and a window of 1000 from 0.08 to 5.
__device__ __noinline__ void chunk_row_again(const ChunkArgs &a, const ChunkSegment &s, int i) {
  const int lane = threadIdx.x & 31;
  const DevLayout &lay = a.lay;
  const bool gqa = lay.kind == KAMERA_GQA;
  const float neg_inf = -__int_as_float(0x7f800000);
  const long long layer0 = (long long)a.layer * a.pool.num_slots;
  const __nv_bfloat16 *pk = a.pool.k + layer0 * lay.row_k + (gqa ? s.kvh * lay.hd : 0);
  const __nv_bfloat16 *pv =
      gqa ? a.pool.v + layer0 * lay.row_v + s.kvh * lay.hd : pk;
  const int vrow = gqa ? lay.row_v : lay.row_k;
  const int col0 = s.part * a.shape.vw, cols = min(a.shape.vw, a.dv - col0);
  int k, h;
  chunk_row(a, s, i, &k, &h);
  const __nv_bfloat16 *q = a.q + (s.row + k) * a.q_stride + (long long)h * a.dk;
  const float c = a.scale * kLog2e;
  float m = neg_inf, l = 0.f, o[8];  // columns lane + 32 e
#pragma unroll
  for (int e = 0; e < 8; ++e) o[e] = 0.f;
  for (int t = first_seen(a, s.first + k); t <= s.first + k; ++t) {
    const int slot = slot_in(a, load_page(a, s.r, t), t);
    if (slot < 0) continue;
    float x = 0.f;
    for (int d = lane; d < a.dk; d += 32)
      x = fmaf(__bfloat162float(q[d]), __bfloat162float(pk[(long long)slot * lay.row_k + d]), x);
    for (int z = 16; z > 0; z >>= 1) x += __shfl_xor_sync(0xffffffffu, x, z);
    x *= c;
    if (x > m) {
      const float f = m == neg_inf ? 0.f : exp2_approx(m - x);
      m = x;
      l *= f;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= f;
    }
    const float p = exp2_approx(x - (m == neg_inf ? 0.f : m));
    l += p;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (lane + 32 * e < cols)
        o[e] = fmaf(p, __bfloat162float(pv[(long long)slot * vrow + col0 + lane + 32 * e]), o[e]);
  }
  const long long rh = (long long)(s.row + k) * a.hq + h;
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (lane + 32 * e < cols)
      a.out[rh * a.dv + col0 + lane + 32 * e] = __float2bfloat16_rn(o[e] * inv);
  if (lane == 0 && s.part == 0) a.lse[rh] = l == 0.f ? neg_inf : (m + log2f(l)) * kLn2;
}

// Worker blockIdx.x's cut block: a warp to a row, the parts' log-sum-exps a lane each, then four
// columns a lane. Then, where an output of the call is not finite, those of the blocks that the
// worker starts which multiply a value that is not finite for a row that does not see it.
__global__ void __launch_bounds__(kJoinThr, 4) chunk_join_kernel(const __grid_constant__ ChunkArgs a) {
  __shared__ ChunkScratch<kJoinThr> found;
  constexpr int kAtOnce = 4;  // rows that a warp joins together, of blocks of two parts
  const int w = blockIdx.x, lane = threadIdx.x & 31;
  const int first = blockIdx.y * (kJoinThr / 32) + (threadIdx.x >> 5);
  const int step = gridDim.y * (kJoinThr / 32);
  const ChunkPlaces places = chunk_places(a.shape, a.ws);
  const float neg_inf = -__int_as_float(0x7f800000);
  ptx::wait_for_previous();
  const ChunkRecord rec = places.rec[w];
  int odd = 0;
  for (int i = threadIdx.x; i < a.shape.n; i += kJoinThr) odd |= places.rec[i].odd;
  odd = __syncthreads_or(odd);
  if (rec.head && !rec.gave_up) {
    const int rb = a.shape.rb, vw = a.shape.vw, np = 1 + rec.more;
    const int cols = min(vw, a.dv - rec.part * vw);
    bool skip = false;
    for (int i = lane; i < rec.more; i += 32) skip |= places.rec[w + 1 + i].gave_up;
    if (!__any_sync(0xffffffffu, skip)) {
      auto place = [&](int p) { return (long long)(2 * (w + p) + (p == 0)) * rb; };
      auto row_of = [&](int i) {  // of q and its head, in out and lse
        const int k = a.pieces > 1 ? 0 : (int)((unsigned)i * a.hpk_magic >> 16);
        return (long long)(rec.row + k) * a.hq + rec.h0 + i - k * a.hpk;
      };
      auto put = [&](long long rh, int col, const float *acc, float inv) {
        uint2 v;
        v.x = pack_bf16(acc[0] * inv, acc[1] * inv);
        v.y = pack_bf16(acc[2] * inv, acc[3] * inv);
        *reinterpret_cast<uint2 *>(a.out + rh * a.dv + rec.part * vw + col) = v;
      };
      for (int i0 = first * kAtOnce; np == 2 && i0 < rec.rows; i0 += step * kAtOnce) {
        // two parts, as most cut blocks have: several rows' loads together
        for (int col = 4 * lane; col < cols; col += 128) {
          float4 v[kAtOnce][2];
          float z[kAtOnce][2];
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const long long at = place(p) + min(i0 + j, rec.rows - 1);
              z[j][p] = places.lse[at];
              v[j][p] = *reinterpret_cast<const float4 *>(places.o + at * vw + col);
            }
#pragma unroll
          for (int j = 0; j < kAtOnce; ++j) {
            if (i0 + j >= rec.rows) break;
            // a part of no mass is left out; a NaN goes on
            const float top = fmaxf(z[j][0], z[j][1]);
            const float f0 = z[j][0] == neg_inf ? 0.f : exp2_approx((z[j][0] - top) * kLog2e);
            const float f1 = z[j][1] == neg_inf ? 0.f : exp2_approx((z[j][1] - top) * kLog2e);
            const float sum = f0 + f1, inv = sum == 0.f ? 0.f : 1.f / sum;
            float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              const float f = p ? f1 : f0;
              if (f == 0.f) continue;
              acc[0] = fmaf(f, v[j][p].x, acc[0]);
              acc[1] = fmaf(f, v[j][p].y, acc[1]);
              acc[2] = fmaf(f, v[j][p].z, acc[2]);
              acc[3] = fmaf(f, v[j][p].w, acc[3]);
            }
            const long long rh = row_of(i0 + j);
            put(rh, col, acc, inv);
            if (col == 0 && rec.part == 0) a.lse[rh] = sum == 0.f ? neg_inf : top + logf(sum);
          }
        }
      }
      for (int i = first; np > 2 && i < rec.rows; i += step) {
        float top = neg_inf;
        for (int p = lane; p < np; p += 32) top = fmaxf(top, places.lse[place(p) + i]);
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        const long long rh = row_of(i);
        for (int col = 0; col < cols; col += 128) {
          const bool in = col + 4 * lane < cols;
          float sum = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
          for (int p0 = 0; p0 < np; p0 += 32) {
            // a part of no mass is left out; a NaN goes on
            const float z = p0 + lane < np ? places.lse[place(p0 + lane) + i] : neg_inf;
            const float wt = z == neg_inf ? 0.f : exp2_approx((z - top) * kLog2e);
            float t = wt;
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            sum += t;
            const int n = min(32, np - p0);
            for (int j0 = 0; j0 < n; j0 += 8) {
              float4 v[8];
#pragma unroll
              for (int j = 0; j < 8; ++j)
                v[j] = in && j0 + j < n
                           ? *reinterpret_cast<const float4 *>(
                                 places.o + (place(p0 + j0 + j) + i) * vw + col + 4 * lane)
                           : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float f = __shfl_sync(0xffffffffu, wt, (j0 + j) & 31);
                if (j0 + j < n && f != 0.f) {
                  acc[0] = fmaf(f, v[j].x, acc[0]);
                  acc[1] = fmaf(f, v[j].y, acc[1]);
                  acc[2] = fmaf(f, v[j].z, acc[2]);
                  acc[3] = fmaf(f, v[j].w, acc[3]);
                }
              }
            }
          }
          const float inv = sum == 0.f ? 0.f : 1.f / sum;
          if (in) put(rh, col + 4 * lane, acc, inv);
          if (lane == 0 && col == 0 && rec.part == 0)
            a.lse[rh] = sum == 0.f ? neg_inf : top + logf(sum);
        }
      }
    }
  }
  if (!odd || rec.gave_up) return;
  const ChunkStart st = chunk_start<kJoinThr>(a, w, &found);
  ChunkWalk walk;
  walk.start(a, st, w);
  ChunkSegment s;
  while (walk.next(a, &s)) {
    const bool again = !s.carry() && chunk_odd(a, s, threadIdx.x >> 5, kJoinThr / 32);
    if (__syncthreads_or(again)) {
      // each row by the warp that has joined it, so that this is what is written last
      const int rows = s.ntok * s.heads, run = s.more == 1 ? kAtOnce : 1;
      for (int i0 = first * run; i0 < rows; i0 += step * run)
        for (int i = i0; i < min(i0 + run, rows); ++i) chunk_row_again(a, s, i);
    }
  }
}

}  // namespace

ChunkShape chunk_shape(const DevLayout &l) {
  if (chunk_tc_layout(l)) return chunk_tc_shape(l);
  const int dv = l.kind == KAMERA_GQA ? l.hd : l.latent;
  return {kRows, kTileSh, (dv + kCols - 1) / kCols, kCols, kSms, 1, 1, 0};
}

void chunk_blocks(ChunkArgs *a, int rows) {
  a->pieces = (a->hpk + rows - 1) / rows;
  a->tb = a->hpk > rows ? 1 : rows / a->hpk;
}

size_t chunk_workspace(const DevLayout &l) { return chunk_places(chunk_shape(l), nullptr).total; }

// How long a wait of the tcgen05 kernels over chunks may take. Tests set it to 0, which makes every
// CTA give up before it begins; not for other use.
extern "C" unsigned long long kamera_chunk_wait_ns;
unsigned long long kamera_chunk_wait_ns = kPrefixWaitNs;

cudaError_t launch_chunk_attention(const ChunkArgs &args, cudaStream_t s) {
  ChunkArgs a = args;
  a.wait_ns = kamera_chunk_wait_ns;
  static int configured[64][4] = {{0}};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const int kind = !chunk_tc_layout(a.lay) ? 0
                   : a.lay.kind == KAMERA_MLA ? 1
                                              : (a.lay.hd == 128 ? 2 : 3);
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev][kind]) {
      e = kind ? prepare_chunk_tc(a.lay)
               : cudaFuncSetAttribute(chunk_gen_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      gen_plan(1024).total);
      if (e != cudaSuccess) return e;
      configured[dev][kind] = 1;
    }
  }
  if (kind) {
    e = launch_chunk_tc(a, s);
  } else {
    chunk_gen_kernel<<<a.shape.n, kThr, gen_plan(a.dk).total, s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  // a warp to a few rows of a cut block
  const long long rows = std::min<long long>(a.shape.rb, (long long)a.n_tokens * a.hpk);
  const int per = kJoinThr / 32 * (rows > 64 ? 4 : 1);
  return launch_early(chunk_join_kernel, dim3(a.shape.n, (unsigned)((rows + per - 1) / per)), kJoinThr,
                      0, s, a);
}

}  // namespace kamera
