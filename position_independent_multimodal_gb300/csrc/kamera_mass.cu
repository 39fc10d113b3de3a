// Attention masses: what the new tokens' softmax weights sum to on each cached token,
//   mass_u = decay mass_u + sum over tokens t that see u, query heads h of exp(s_thu - lse_th),
// with the scores taken again from Q and K and the log-sum-exp that attention left. The kernel of
// the layouts that the tcgen05 kernel (kamera_mass_tc.cu) does not take, and the join of the blocks
// that workers cut.
//
// mass_gen_kernel: S^T = K Q^T by m16n8k16 products on registers, four warps of 16 cached tokens
// against tiles of 32 query rows, so that a token's sum stays in a thread's register over all the
// query rows. Products, weights and sums are float32. Bound as chunk_gen_kernel: 27 TFLOP/s over 4
// requests of 500 tokens over 4000 (16 query heads, 4 KV heads of 96), 32 that decode over 4000 in 153 us.
#include <mutex>

#include "kamera_mass.cuh"
#include "kamera_mma.cuh"
#include "kamera_ptx.cuh"

namespace kamera {

namespace {

constexpr int kToks = 64, kQ = 32, kThr = 128;

__host__ __device__ inline int gen_smem(int dk) { return (kToks + kQ) * (2 * dk + 16); }

__global__ void __launch_bounds__(kThr) mass_gen_kernel(const __grid_constant__ MassArgs a) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ ChunkScratch<kThr> found;
  __shared__ int slots[kToks], see0[kQ], see1[kQ];
  __shared__ float base[kQ];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, w = blockIdx.x;
  const ChunkArgs &b = a.b;
  const DevLayout &lay = b.lay;
  const int pitch = 2 * b.dk + 16, qp = b.dk >> 3;
  const uint32_t sk = ptx::smem_addr(smem), sq = sk + kToks * pitch;
  const MassPlaces places = mass_places(a.shape, a.ws);
  const __nv_bfloat16 *pk = b.pool.k + (long long)b.layer * b.pool.num_slots * lay.row_k;
  const float neg_inf = -__int_as_float(0x7f800000);
  const float c = b.scale * kLog2e;
  const ChunkStart st = mass_start<kThr>(a, w, &found);
  ptx::launch_dependents();
  MassWalk walk;
  walk.start(a, st, w);
  MassSegment s = {};
  int segments = 0;
  for (; walk.next(a, &s); ++segments) {
    // the first token that the first of the block's new tokens sees: none before it is looked at
    const int lo = first_seen(b, s.q.past + s.i0 * b.tb);
    __syncthreads();
    if (tid < kToks) {
      const int tok = s.tok0 + tid;
      slots[tid] = tok >= lo && tok < s.q.ctx ? slot_in(b, load_page(b, s.r, tok), tok) : -1;
    }
    float sum[2] = {0.f, 0.f};
    int had = -1;  // KV head of the rows in shared memory
    for (int k = s.k0; k < s.k1; ++k) {
      const int hp = k / s.ni, i = s.i0 + k - hp * s.ni, piece = hp % b.pieces, kvh = hp / b.pieces;
      const int h0 = kvh * b.hpk + piece * a.shape.qr;
      const int heads = min(b.hpk - piece * a.shape.qr, a.shape.qr);
      const int rows = heads * min(b.tb, s.q.n - i * b.tb);
      __syncthreads();
      if (kvh != had) {
        const int kcol = lay.kind == KAMERA_GQA ? kvh * lay.hd : 0;
        for (int e = tid; e < kToks * qp; e += kThr) {
          const int t = e / qp, p = e - t * qp, slot = slots[t];
          ptx::cp_async16(sk + t * pitch + 16 * p,
                          slot >= 0 ? pk + (long long)slot * lay.row_k + kcol + 8 * p : pk,
                          slot >= 0 ? 16u : 0u);
        }
        had = kvh;
      }
      auto place = [&](int y, int *tok, int *h) {  // of row y: its new token, its query head
        const int d = b.pieces > 1 ? 0 : (int)((unsigned)y * b.hpk_magic >> 16);
        *tok = i * b.tb + d;
        *h = h0 + y - d * b.hpk;
      };
      for (int e = tid; e < kQ * qp; e += kThr) {
        const int y = e / qp, p = e - y * qp;
        int tok, h;
        place(y < rows ? y : 0, &tok, &h);
        ptx::cp_async16(sq + y * pitch + 16 * p,
                        b.q + (s.q.row + tok) * b.q_stride + (long long)h * b.dk + 8 * p,
                        y < rows ? 16u : 0u);
      }
      ptx::cp_async_commit();
      if (tid < kQ) {
        int tok, h;
        place(tid < rows ? tid : 0, &tok, &h);
        const float z = a.lse[(long long)(s.q.row + tok) * b.hq + h];
        // of a row that saw nothing (and of none) nothing is laid on any token
        const bool on = tid < rows && z != neg_inf;
        base[tid] = z * kLog2e;
        see0[tid] = on ? first_seen(b, s.q.past + tok) : 0x7FFFFFFF;
        see1[tid] = on ? s.q.past + tok + 1 : 0;
      }
      ptx::cp_async_wait_all();
      __syncthreads();
      float x[kQ / 8][4];
#pragma unroll
      for (int n = 0; n < kQ / 8; ++n)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[n][e] = 0.f;
      for (int d = 0; d < b.dk; d += 16) {
        uint32_t ka[4];
        ldsm4(sk + (16 * warp + (lane & 15)) * pitch + 2 * d + 16 * (lane >> 4), ka);
#pragma unroll
        for (int n = 0; n < kQ / 16; ++n) {
          uint32_t qb[4];
          ldsm4(sq + (16 * n + (lane & 7) + ((lane >> 4) << 3)) * pitch + 2 * d +
                    16 * ((lane >> 3) & 1), qb);
          mma16816(x[2 * n], ka, qb[0], qb[1]);
          mma16816(x[2 * n + 1], ka, qb[2], qb[3]);
        }
      }
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        const int t = 16 * warp + 8 * y + (lane >> 2);
        const bool have = slots[t] >= 0;
#pragma unroll
        for (int n = 0; n < kQ / 8; ++n)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = 8 * n + 2 * (lane & 3) + e;
            const bool on = have && s.tok0 + t >= see0[j] && s.tok0 + t < see1[j];
            sum[y] += on ? exp2_approx(fmaf(x[n][2 * y + e], c, -base[j])) : 0.f;
          }
      }
    }
#pragma unroll
    for (int y = 0; y < 2; ++y) {
      sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 1);
      sum[y] += __shfl_xor_sync(0xffffffffu, sum[y], 2);
      if ((lane & 3) == 0) mass_out(a, places, s, w, 16 * warp + 8 * y + (lane >> 2), sum[y]);
    }
  }
  if (tid == 0) mass_note(places.rec + w, s, segments, false);
}

// ---------------------------------------------------------------------------------------
// join
// ---------------------------------------------------------------------------------------

constexpr int kJoinThr = 256;

// Worker blockIdx.x's cut block, its parts added in the workers' order; and of every n-th request
// the tokens that no new token sees, whose masses only fade.
__global__ void __launch_bounds__(kJoinThr) mass_join_kernel(const __grid_constant__ MassArgs a) {
  const int w = blockIdx.x, kt = a.shape.kt;
  const MassPlaces places = mass_places(a.shape, a.ws);
  ptx::wait_for_previous();
  const MassRecord rec = places.rec[w];
  if (rec.head) {
    int skip = rec.gave_up;
    for (int i = threadIdx.x; i < rec.more; i += kJoinThr) skip |= places.rec[w + 1 + i].gave_up;
    const int ctx = a.b.ctx_len[rec.r];
    if (!__syncthreads_or(skip)) {
      for (int i = threadIdx.x; i < kt && rec.tok0 + i < ctx; i += kJoinThr) {
        float sum = places.sum[(2ll * w + 1) * kt + i];
        for (int p = 1; p <= rec.more; ++p) sum += places.sum[2ll * (w + p) * kt + i];
        float *m = a.mass + (long long)rec.r * a.mass_stride + rec.tok0 + i;
        *m = a.decay == 0.f ? sum : fmaf(a.decay, *m, sum);
      }
    }
  }
  if (a.b.window == 0 || a.decay == 1.f) return;
  int bad = 0;
  for (int r = threadIdx.x; r < a.b.n_reqs; r += kJoinThr) {
    bool bs, bi;
    chunk_request(a.b, r, &bs, &bi);
    bad |= bs;
  }
  if (__syncthreads_or(bad)) return;
  for (int r = w; r < a.b.n_reqs; r += gridDim.x) {
    bool bs, bi;
    const ChunkRequest q = chunk_request(a.b, r, &bs, &bi);
    if (q.n == 0) continue;
    const int end = mass_tile0(a, q) * kt;
    for (int i = threadIdx.x; i < end; i += kJoinThr) {
      float *m = a.mass + (long long)r * a.mass_stride + i;
      *m = a.decay == 0.f ? 0.f : a.decay * *m;
    }
  }
}

}  // namespace

MassShape mass_shape(const DevLayout &l) {
  return chunk_tc_layout(l) ? mass_tc_shape(l) : MassShape{kToks, kQ, kSms};
}

size_t mass_workspace(const DevLayout &l) { return mass_places(mass_shape(l), nullptr).total; }

extern "C" unsigned long long kamera_chunk_wait_ns;  // kamera_chunk.cu

cudaError_t launch_attention_mass(const MassArgs &args, cudaStream_t s) {
  MassArgs a = args;
  a.b.wait_ns = kamera_chunk_wait_ns;
  static int configured[64][4] = {{0}};
  static std::mutex mu;
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  const DevLayout &l = a.b.lay;
  const int kind = !chunk_tc_layout(l) ? 0 : l.kind == KAMERA_MLA ? 1 : (l.hd == 128 ? 2 : 3);
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev][kind]) {
      e = kind ? prepare_mass_tc(l)
               : cudaFuncSetAttribute(mass_gen_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                      gen_smem(1024));
      if (e != cudaSuccess) return e;
      configured[dev][kind] = 1;
    }
  }
  if (kind) {
    e = launch_mass_tc(a, s);
  } else {
    mass_gen_kernel<<<a.shape.n, kThr, gen_smem(a.b.dk), s>>>(a);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return e;
  return launch_early(mass_join_kernel, dim3(a.shape.n), kJoinThr, 0, s, a);
}

}  // namespace kamera
