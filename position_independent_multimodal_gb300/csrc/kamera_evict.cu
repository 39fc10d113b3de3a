// Eviction: of each listed request the first tokens, the last ones and those of the greatest mass
// stay and are drawn together in order, in every layer.
//
//  * evict_pick_kernel, a CTA to a request: the mass of the last token that stays is found by three
//    rounds of counting (11, 11 and 10 bits of the masses' order), then every warp lists what stays
//    of its part of the tokens, in order. Ties go to the lowest token. The masses are read six times
//    from L2 by one SM: 10 us for 701 tokens, 13 for 20 requests of 4000, 40 for six of 30000, next
//    to 15, 552 and 335 of the moves. It is bound by its instructions (equal masses of a warp counted
//    as one by a match: 54 us for 40).
//  * evict_move_kernel: token kept[j] moves to token j <= kept[j]. A CTA takes one strip of columns
//    of one layer and walks the tokens upwards, several stages of rows on their way through shared
//    memory: rows are written only after all rows up to them have been read, and what later stages
//    read lies above all that has been written, so reads may run ahead of the writes. The masses
//    move likewise. It is bound by HBM: 3.76 GB of rows of 512 columns read and written in 552 us, 6.8
//    TB/s, as fast as a copy; 2.1 GB of MLA's, whose 816 strips do not fill the last round of CTAs, in
//    335 us, 6.2 TB/s. Two, three and five stages of 64 rows on their way: 395, 388 and 399 us of the
//    call for MLA; strips of 128 bytes 393 to 401, and 604 to 616 of the call for 582 at 20 requests.
#include <mutex>

#include "kamera_dev.cuh"
#include "kamera_ptx.cuh"

namespace kamera {

namespace {

// What the first kernel leaves of an item for the second.
struct EvictPlan {
  int n, keep;   // its tokens, those that stay
  int from;      // the first that moves; keep: nothing does
  int req;
};

// Masses in their order: a greater mass has a greater key; NaN is above all, -0 is 0.
__device__ __forceinline__ uint32_t mass_key(float x) {
  if (x != x) return 0xffffffffu;
  const uint32_t u = __float_as_uint(x + 0.f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

constexpr int kPickThr = 1024, kBins = 2048;
constexpr int kLoads = 8;  // masses that a thread asks for together

__global__ void __launch_bounds__(kPickThr) evict_pick_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ int bins[kBins], sums[32], chosen[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, ps = a.lay.page_size;
  ptx::launch_dependents();
  const kamera_evict_item it = a.items[blockIdx.x];
  EvictPlan *plan = static_cast<EvictPlan *>(a.ws) + blockIdx.x;
  const int n = it.num_tokens, k = min(it.keep, n);
  const bool ok = it.req >= 0 && it.req < a.pool.num_reqs && n >= 0 &&
                  n <= (long long)a.pool.pt_stride * ps && n <= a.mass_stride && it.first >= 0 &&
                  it.last >= 0 && it.keep >= 0 && (long long)it.first + it.last <= it.keep &&
                  k <= a.kept_stride;
  if (!ok) {
    if (tid == 0) {
      atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
      *plan = {0, 0, 0, 0};
    }
    return;
  }
  const int *pages = a.pool.pt + (long long)it.req * a.pool.pt_stride;
  int *kept = a.kept + (long long)blockIdx.x * a.kept_stride;
  if (k == n) {  // all stay
    for (int i = tid; i < n; i += kPickThr) kept[i] = i;
    if (tid == 0) *plan = {n, n, n, it.req};
    return;
  }
  const float *mass = a.mass + (long long)it.req * a.mass_stride;
  const int c0 = it.first, c1 = n - it.last;  // the tokens that are judged
  auto of_warps_before = [&]() {
    return __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0);
  };
  // the smallest key that stays, found from its upper bits down, and how many of that key stay
  uint32_t key = 0;
  int need = k - it.first - it.last;
  if (need > 0) {
#pragma unroll 1
    for (int round = 0; round < 3; ++round) {
      const int shift = round == 0 ? 21 : round == 1 ? 10 : 0, bits = round == 2 ? 10 : 11;
      for (int i = tid; i < kBins; i += kPickThr) bins[i] = 0;
      __syncthreads();
      for (int i0 = c0 + tid; i0 < c1; i0 += kLoads * kPickThr) {
        float m[kLoads];
#pragma unroll
        for (int e = 0; e < kLoads; ++e)
          m[e] = i0 + e * kPickThr < c1 ? mass[i0 + e * kPickThr] : 0.f;
#pragma unroll
        for (int e = 0; e < kLoads; ++e) {
          const uint32_t x = mass_key(m[e]);
          if (i0 + e * kPickThr < c1 &&
              (round == 0 || x >> (shift + bits) == key >> (shift + bits)))
            atomicAdd(bins + (x >> shift & ((1u << bits) - 1u)), 1);
        }
      }
      __syncthreads();
      // bins from the greatest down: thread t has bins kBins - 1 - 2 t and the one below
      const int b0 = bins[kBins - 1 - 2 * tid], b1 = bins[kBins - 2 - 2 * tid];
      int incl = b0 + b1;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane == 31) sums[warp] = incl;
      __syncthreads();
      const int before = incl - b0 - b1 + of_warps_before();
      if (before < need && before + b0 + b1 >= need) {
        const bool low = before + b0 < need;
        chosen[0] = kBins - 1 - 2 * tid - low;
        chosen[1] = need - before - (low ? b0 : 0);
      }
      __syncthreads();
      key |= (uint32_t)chosen[0] << shift;
      need = chosen[1];
      __syncthreads();
    }
  }
  // Each warp has a run of tokens: its ties, then (with the ties before it) what it keeps.
  const int per = ((n + 31) / 32 + 31) & ~31, t0 = min(n, warp * per), t1 = min(n, t0 + per);
  const bool judged = k > it.first + it.last;
  auto state = [&](int t, float m) {  // 0 goes, 1 a tie, 2 stays
    if (t >= t1) return 0;
    if (t < c0 || t >= c1) return 2;
    if (!judged) return 0;
    const uint32_t x = mass_key(m);
    return x > key ? 2 : (x == key ? 1 : 0);
  };
  // calls f(token of the lane, its state) for the warp's tokens, 32 at a time
  auto each = [&](auto f) {
    for (int t = t0 + lane; t - lane < t1; t += 32 * kLoads) {
      float m[kLoads];
#pragma unroll
      for (int e = 0; e < kLoads; ++e) {
        const int u = t + 32 * e;
        m[e] = judged && u < t1 && u >= c0 && u < c1 ? mass[u] : 0.f;
      }
#pragma unroll
      for (int e = 0; e < kLoads; ++e)
        if (t - lane + 32 * e < t1) f(t + 32 * e, state(t + 32 * e, m[e]));
    }
  };
  int ties = 0, sure = 0;
  each([&](int, int v) {
    ties += __popc(__ballot_sync(0xffffffffu, v == 1));
    sure += __popc(__ballot_sync(0xffffffffu, v == 2));
  });
  if (lane == 0) sums[warp] = ties;
  __syncthreads();
  const int tie0 = of_warps_before();
  __syncthreads();
  const int mine = sure + max(0, min(ties, need - tie0));
  if (lane == 0) sums[warp] = mine;
  if (tid == 0) chosen[0] = k;
  __syncthreads();
  const int at = of_warps_before();
  int from = k;  // the first token that moves
  int *list = kept;
  // what stays is listed, unless pages forbid it: so the first token that moves is found first
  for (int pass = 0; pass < 2; ++pass) {
    int j = at, tie = tie0;
    each([&](int t, int v) {
      const uint32_t eq = __ballot_sync(0xffffffffu, v == 1), below = (1u << lane) - 1u;
      const bool stays = v == 2 || (v == 1 && tie + __popc(eq & below) < need);
      const uint32_t in = __ballot_sync(0xffffffffu, stays);
      const int to = j + __popc(in & below);
      if (stays) {
        if (pass == 0) {
          if (to != t) from = min(from, to);
        } else {
          list[to] = t;
        }
      }
      j += __popc(in);
      tie += __popc(eq);
    });
    if (pass == 1) break;
    for (int o = 16; o > 0; o >>= 1) from = min(from, __shfl_xor_sync(0xffffffffu, from, o));
    if (lane == 0 && from < k) atomicMin(chosen, from);
    __syncthreads();
    from = chosen[0];
    bool outside = false, shared = false;
    for (int p = tid; p < (int)(((long long)n + ps - 1) / ps); p += kPickThr) {
      const int page = pages[p];
      const bool out = page < 0 || ((long long)page + 1) * ps > a.pool.num_slots;
      outside |= out;
      // a page that is written must be the request's alone
      if (!out && from < k && (long long)(p + 1) * ps > from && (long long)p * ps < k)
        shared |= a.refs[page] > 1;
    }
    if (outside) atomicOr(a.status, KAMERA_DEVICE_SLOT_OOB);
    if (shared) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
    if (__syncthreads_or(outside || shared)) {
      if (tid == 0) *plan = {0, 0, 0, 0};
      return;
    }
  }
  if (tid == 0) *plan = {n, k, from, it.req};
}

// ---------------------------------------------------------------------------------------
// rows
// ---------------------------------------------------------------------------------------

constexpr int kMoveThr = 256;
constexpr int kAhead = 3;                          // stages of rows on their way
constexpr int kStages = kAhead + 1, kLists = kAhead + 2;
constexpr int kPieces = 16;                        // 16-byte pieces of a strip
constexpr int kStageRows = 64;
constexpr int kStageBytes = kStageRows * kPieces * 16;

__global__ void __launch_bounds__(kMoveThr) evict_move_kernel(const __grid_constant__ EvictArgs a,
                                                              int strips_k, int strips) {
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ int rows_at[kLists][2][kStageRows];  // slots that rows come from, go to
  const int tid = threadIdx.x, ps = a.lay.page_size;
  ptx::wait_for_previous();
  const EvictPlan plan = static_cast<const EvictPlan *>(a.ws)[blockIdx.y];
  if (plan.from >= plan.keep && plan.keep == plan.n) return;
  const int *kept = a.kept + (long long)blockIdx.y * a.kept_stride;
  if ((int)blockIdx.x == strips * a.lay.L) {  // the masses
    float *mass = a.mass + (long long)plan.req * a.mass_stride;
    for (int j = plan.from; j < plan.keep; j += kMoveThr) {
      const bool in = j + tid < plan.keep;
      const float v = in ? mass[kept[j + tid]] : 0.f;
      __syncthreads();
      if (in) mass[j + tid] = v;
      __syncthreads();
    }
    for (int j = plan.keep + tid; j < plan.n; j += kMoveThr) mass[j] = 0.f;
    return;
  }
  const int layer = blockIdx.x / strips, strip = blockIdx.x - layer * strips;
  const bool is_k = strip < strips_k;
  const int row = is_k ? a.lay.row_k : a.lay.row_v;
  const int p0 = (is_k ? strip : strip - strips_k) * kPieces, np = min(kPieces, row / 8 - p0);
  __nv_bfloat16 *base = (is_k ? a.pool.k : a.pool.v) +
                        (long long)layer * a.pool.num_slots * row + p0 * 8;
  const int *pages = a.pool.pt + (long long)plan.req * a.pool.pt_stride;
  const int stages = (plan.keep - plan.from + kStageRows - 1) / kStageRows;
  const uint32_t sb = ptx::smem_addr(smem);
  // The rows of a stage, a thread to the slot that one comes from or goes to. Its token and its page
  // are asked for a stage ahead each, so no stage waits for them.
  const int part = tid / kStageRows, mine = tid & (kStageRows - 1);
  int tok = 0, was = 0, page = 0, tok_of = 0, page_of = 0;  // stages with a token, with a page
  auto look_up = [&](bool list) {
    if (part > 1) return;
    if (list) {
      rows_at[(page_of - 1) % kLists][part][mine] = page * ps + was % ps;
    }
    if (page_of < tok_of) {
      was = tok;
      page = pages[tok / ps];
      ++page_of;
    }
    const int j = min(plan.from + tok_of * kStageRows + mine, plan.keep - 1);
    tok = part ? j : kept[j];
    ++tok_of;
  };
  auto rows_of = [&](int st) { return min(kStageRows, plan.keep - plan.from - st * kStageRows); };
  auto read = [&](int st) {
    if (st < stages) {
      const int b = st % kStages, rows = rows_of(st);
      for (int e = tid; e < kStageRows * kPieces; e += kMoveThr) {
        const int i = e / kPieces, p = e % kPieces;
        if (i < rows && p < np)
          ptx::cp_async16(sb + b * kStageBytes + e * 16,
                          base + (long long)rows_at[st % kLists][0][i] * row + p * 8, 16u);
      }
    }
    ptx::cp_async_commit();
  };
  if (stages == 0) return;
  look_up(false);                                      // tokens of stage 0
  look_up(false);                                      // its pages, tokens of stage 1
  for (int k = 0; k <= kAhead; ++k) look_up(true);     // lists of stages 0 to kAhead
  __syncthreads();
  for (int k = 0; k < kAhead; ++k) read(k);
  for (int st = 0; st < stages; ++st) {
    read(st + kAhead);
    look_up(true);                                     // of stage st + kAhead + 1
    ptx::cp_async_wait_group<kAhead>();
    __syncthreads();  // the stage has been read by all
    const int b = st % kStages, rows = rows_of(st);
    for (int e = tid; e < kStageRows * kPieces; e += kMoveThr) {
      const int i = e / kPieces, p = e % kPieces;
      if (i < rows && p < np)
        *reinterpret_cast<uint4 *>(base + (long long)rows_at[st % kLists][1][i] * row + p * 8) =
            *reinterpret_cast<const uint4 *>(smem + b * kStageBytes + e * 16);
    }
    __syncthreads();
  }
}

}  // namespace

size_t evict_workspace(int n) { return sizeof(EvictPlan) * (size_t)n; }

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t s) {
  evict_pick_kernel<<<a.n, kPickThr, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  const int strips_k = (a.lay.row_k / 8 + kPieces - 1) / kPieces;
  const int strips = strips_k + (a.lay.kind == KAMERA_GQA ? (a.lay.row_v / 8 + kPieces - 1) / kPieces : 0);
  static int configured[64] = {0};
  static std::mutex mu;
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      e = cudaFuncSetAttribute(evict_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               kStages * kStageBytes);
      if (e != cudaSuccess) return e;
      configured[dev] = 1;
    }
  }
  return launch_early(evict_move_kernel, dim3(strips * a.lay.L + 1, a.n), kMoveThr,
                      kStages * kStageBytes, s, a, strips_k, strips);
}

}  // namespace kamera
