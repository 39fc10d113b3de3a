// Work division of attention over chunks of new tokens, used by its kernels.
//
// Each request's new tokens are the last of its context; token t sees tokens [0, t], or the last
// `window` of them. A block is a run of tb consecutive new tokens of a request with the query
// heads of one KV head (and one part of V's columns): at most rb query rows that read the same
// rows of K and V. A block's work is its tiles of 2^tile_sh cached tokens, from the first that a row of
// it sees to the last. It counts in units: some for each tile, more where the block has more rows than
// fill a tensor-core tile, and some for its start and end. Units are numbered by request, KV head,
// block, tile; workers take consecutive ones, as many as one another, whatever the lengths, and cut at
// most their first and last block, between tiles. Blocks that one worker has whole
// are written at once. Of a cut block the worker of its first tile writes its part to the worker's
// home place and the others theirs to their carry places; the join kernel merges them by their
// log-sum-exp.
//
// No plan is made ahead: a request's units are counted by a closed form (sums of rounded linear
// terms), so every CTA finds its first block by itself in one pass over the requests.
#pragma once

#include "kamera_prefix.cuh"

namespace kamera {

// What a worker leaves for the join kernel.
struct ChunkRecord {
  int head;        // 1: its last segment is the first part of a cut block
  int more;        // of that block: workers that follow on it
  int row, rows;   // of it: row of q of its first token, query rows
  int h0, part;    // of it: first query head, part of V's columns
  int gave_up;
  int odd;         // 1: some of its outputs are not finite
  int pad[8];
};

struct ChunkPlaces {
  ChunkRecord *rec;   // [n]
  float *lse;         // [n][2][rb]: carry, home
  float *o;           // [n][2][rb][vw]
  size_t total;
};

__host__ __device__ inline ChunkPlaces chunk_places(const ChunkShape &s, void *ws) {
  ChunkPlaces p;
  const size_t skew = static_cast<size_t>(-reinterpret_cast<intptr_t>(ws)) & 127;
  unsigned char *b = static_cast<unsigned char *>(ws) + skew;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    unsigned char *at = b + o;
    o += (bytes + 127) & ~static_cast<size_t>(127);
    return at;
  };
  p.rec = reinterpret_cast<ChunkRecord *>(take(sizeof(ChunkRecord) * s.n));
  p.lse = reinterpret_cast<float *>(take(8ull * s.n * s.rb));
  p.o = reinterpret_cast<float *>(take(8ull * s.n * s.rb * s.vw));
  p.total = o + 112;  // the workspace is 16-byte aligned
  return p;
}

// Sum over i < n of floor((a i + b) / m), by Euclid's steps on (m, a); a n + b < 2^32, m > 0.
__device__ __forceinline__ long long floor_sum(unsigned n, unsigned m, unsigned a, unsigned b) {
  long long sum = 0;
  while (n > 0) {
    sum += (long long)(n & 1 ? (n - 1) / 2 : n / 2) * (n & 1 ? n : n - 1) * (a / m) +
           (long long)n * (b / m);
    a %= m;
    b %= m;
    const unsigned y = a * n + b;
    n = y / m;
    b = y - n * m;
    const unsigned t = a;
    a = m;
    m = t;
  }
  return sum;
}

// A request of the call.
struct ChunkRequest {
  int row, n;       // its first row of q, its new tokens (0: nothing to do)
  int ctx, past;    // its context, the part before the new tokens
  int nb;           // blocks of tokens
};

template <class Args>
__device__ __forceinline__ ChunkRequest chunk_request(const Args &a, int r, bool *bad_start,
                                                      bool *bad_item) {
  ChunkRequest q;
  q.row = a.token_start[r];
  const int end = a.token_start[r + 1];
  q.ctx = a.ctx_len[r];
  q.n = end - q.row;
  *bad_start = q.row < 0 || end < q.row || end > a.n_tokens;
  if (*bad_start) q.n = 0;
  *bad_item = q.n > 0 && (q.ctx < q.n || q.ctx > a.max_ctx);
  if (*bad_item) q.n = 0;
  q.past = q.ctx - q.n;
  q.nb = ceil_div(q.n, a.tb);
  return q;
}

// First token seen by the token at `tok`.
template <class Args>
__device__ __forceinline__ int first_seen(const Args &a, int tok) {
  return a.window > 0 && tok >= a.window ? tok - a.window + 1 : 0;
}

// Tiles of a request's first j blocks.
__device__ __forceinline__ long long chunk_tiles(const ChunkArgs &a, const ChunkRequest &q, int j) {
  const int sh = a.shape.tile_sh;
  const unsigned m = 1u << sh, up = m - 1u;
  long long sum = 0;
  int whole = j;
  if (j == q.nb) {  // the last one may have fewer tokens
    --whole;
    sum += ((unsigned)q.ctx + up) >> sh;
  }
  sum += floor_sum(whole, m, a.tb, (unsigned)q.past + a.tb + up);
  if (a.window > 0) {
    const int lead = a.window - 1 - q.past;  // blocks that start before it see from token 0 on
    const int i0 = lead > 0 ? ceil_div(lead, a.tb) : 0;
    if (j > i0) sum -= floor_sum(j - i0, m, a.tb, (unsigned)(q.past + i0 * a.tb - (a.window - 1)));
  }
  return sum;
}

// Units of a tile of a block of `ntok` tokens.
__device__ __forceinline__ int chunk_weight(const ChunkArgs &a, int ntok) {
  return a.pieces > 1 || ntok * a.hpk > a.shape.rb >> 1 ? a.shape.wide : a.shape.thin;
}
// Units of a request's first j blocks, of one KV head (and piece, and part of V's columns).
__device__ __forceinline__ long long chunk_units(const ChunkArgs &a, const ChunkRequest &q, int j) {
  const int w = chunk_weight(a, a.tb);
  long long sum = w * chunk_tiles(a, q, j) + (long long)a.shape.extra * j;
  if (j == q.nb) {  // the last one may have fewer tokens
    const int first = (q.nb - 1) * a.tb, sh = a.shape.tile_sh;
    const int tiles = (int)(((unsigned)q.ctx + (1u << sh) - 1u) >> sh) -
                      (first_seen(a, q.past + first) >> sh);
    sum += (long long)(chunk_weight(a, q.n - first) - w) * tiles;
  }
  return sum;
}
// The tile of a block that its unit u is of, with w units to a tile; a block's first units, for its
// start and end, go with its first tile.
__device__ __forceinline__ int chunk_tile(const ChunkArgs &a, int u, int w) {
  return max(u - a.shape.extra, 0) / w;
}

// Where a worker starts, found by all threads of the CTA.
struct ChunkStart {
  long long quot, rem;   // units of the call / workers and the rest
  long long units;       // of this worker
  long long off;         // of its first unit in its request
  int r;                 // that request
  int bad;               // the call's token_start is no such list: nothing is done
};

template <int THR>
struct ChunkScratch {
  long long sums[THR / 32];
  long long off;
  int r;
};

// `units_of`: a request's units. `a`: the batch, `workers`: at most; each has `least` units or more.
template <int THR, class Units>
__device__ __forceinline__ ChunkStart units_start(const ChunkArgs &a, int workers, int least,
                                                  int worker, ChunkScratch<THR> *sh,
                                                  Units units_of) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_reqs + THR - 1) / THR;
  const int r0 = min(a.n_reqs, tid * per), r1 = min(a.n_reqs, r0 + per);
  bool bad = false, bad_item = false;
  long long mine = 0;
  for (int r = r0; r < r1; ++r) {
    bool bs, bi;
    const ChunkRequest q = chunk_request(a, r, &bs, &bi);
    bad |= bs;
    bad_item |= bi;
    if (q.n) mine += units_of(q);
  }
  long long incl = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sh->sums[warp] = incl;
  if (worker == 0 && (bad || bad_item)) atomicOr(a.status, KAMERA_DEVICE_BAD_ITEM);
  ChunkStart s;
  s.bad = __syncthreads_or(bad);
  long long before = 0, total = 0;
  for (int i = 0; i < THR / 32; ++i) {
    if (i < warp) before += sh->sums[i];
    total += sh->sums[i];
  }
  if (s.bad) total = 0;
  const int n = total < (long long)workers * least ? max((int)total / least, 1) : workers;
  s.quot = div_pos(total, n);
  s.rem = total - s.quot * n;
  const long long u0 = first_unit(s.quot, s.rem, min(worker, n));
  s.units = first_unit(s.quot, s.rem, min(worker + 1, n)) - u0;
  const long long excl = before + incl - mine;
  if (s.units > 0 && u0 >= excl && u0 < excl + mine) {
    long long off = u0 - excl;
    for (int r = r0; r < r1; ++r) {
      bool bs, bi;
      const ChunkRequest q = chunk_request(a, r, &bs, &bi);
      const long long u = q.n ? units_of(q) : 0;
      if (off < u) {
        sh->off = off;
        sh->r = r;
        break;
      }
      off -= u;
    }
  }
  __syncthreads();
  s.off = sh->off;
  s.r = sh->r;
  return s;
}

template <int THR>
__device__ __forceinline__ ChunkStart chunk_start(const ChunkArgs &a, int worker,
                                                  ChunkScratch<THR> *sh) {
  return units_start<THR>(a, a.shape.n, a.shape.wide, worker, sh, [&](const ChunkRequest &q) {
    return (long long)a.n_kv * a.pieces * a.shape.vh * chunk_units(a, q, q.nb);
  });
}

// A run of tiles of one block, as a worker takes it.
struct ChunkSegment {
  int r;               // the request
  int row, ntok;       // row of q of the block's first token, its tokens
  int first, ctx;      // that token's place in the context, the context
  int h0, heads;       // first query head, query heads of each token
  int kvh, part;       // KV head, part of V's columns
  int t0, t1;          // tiles
  int more;            // -1: starts inside its block; else workers that follow on the block

  __device__ __forceinline__ bool carry() const { return more < 0; }
};

// Walks a worker's segments; by whole warps.
struct ChunkWalk {
  ChunkRequest q;
  long long left, quot, rem;
  int r, hb, j, u, worker;  // the next block (request, head x part, block), its next unit

  __device__ __forceinline__ void start(const ChunkArgs &a, const ChunkStart &s, int worker_) {
    worker = worker_;
    left = s.units;
    quot = s.quot;
    rem = s.rem;
    r = s.r;
    if (left == 0) return;
    bool bs, bi;
    q = chunk_request(a, r, &bs, &bi);
    const long long per = chunk_units(a, q, q.nb);
    const long long h = div_pos(s.off, per), rest = s.off - h * per;
    hb = (int)h;
    const int lane = threadIdx.x & 31;
    j = 0;  // the last block that starts at or before `rest`
    for (int len = q.nb; len > 1;) {
      const int step = (len + 31) >> 5, k = j + lane * step;
      const bool in = lane * step < len && (lane == 0 || chunk_units(a, q, k) <= rest);
      const int i = __popc(__ballot_sync(0xffffffffu, in)) - 1;
      j += i * step;
      len = step == 1 ? 1 : min(step, len - i * step);
    }
    u = (int)(rest - (j ? chunk_units(a, q, j) : 0));
  }
  // The next segment, which has a tile: a cut between two units of one tile is before that tile, so a
  // worker may have units of a block and no tile of it, at its end alone: with `wide` units or more a
  // worker that begins behind a block's first tile has one.
  __device__ __forceinline__ bool next(const ChunkArgs &a, ChunkSegment *s) {
    while (left > 0)
      if (step(a, s)) return true;
    return false;
  }
  __device__ __forceinline__ bool step(const ChunkArgs &a, ChunkSegment *s) {
    const int heads = a.n_kv * a.pieces * a.shape.vh;
    if (hb == heads) {
      do {
        bool bs, bi;
        q = chunk_request(a, ++r, &bs, &bi);
      } while (q.n == 0);
      hb = j = u = 0;
    }
    const int part = hb % a.shape.vh, hp = hb / a.shape.vh, piece = hp % a.pieces;
    const int sh = a.shape.tile_sh;
    s->r = r;
    s->kvh = hp / a.pieces;
    s->part = part;
    s->h0 = s->kvh * a.hpk + piece * a.shape.rb;
    s->heads = min(a.hpk - piece * a.shape.rb, a.shape.rb);
    s->row = q.row + j * a.tb;
    s->ntok = min(a.tb, q.n - j * a.tb);
    s->first = q.past + j * a.tb;
    s->ctx = q.ctx;
    const int b0 = first_seen(a, s->first) >> sh;
    const int b1 = (int)(((unsigned)(s->first + s->ntok) + (1u << sh) - 1u) >> sh);
    const int w = chunk_weight(a, s->ntok), all = (b1 - b0) * w + a.shape.extra;
    const int end = left < all - u ? u + (int)left : all;
    const int t0 = chunk_tile(a, u, w), t1 = chunk_tile(a, end, w);
    s->t0 = b0 + t0;
    s->t1 = b0 + t1;
    s->more = t0 > 0 ? -1 : end < all ? workers_for(quot, rem, worker + 1, all - end) : 0;
    left -= end - u;
    u = 0;
    if (++j == q.nb) {
      j = 0;
      ++hb;
    }
    return t0 < t1;
  }
};

// Token of row i of a block (its place among the block's) and the row's head.
__device__ __forceinline__ void chunk_row(const ChunkArgs &a, const ChunkSegment &s, int i,
                                          int *tok, int *h) {
  const int k = a.pieces > 1 ? 0 : (int)((unsigned)i * a.hpk_magic >> 16);  // i / hpk for i < 256
  *tok = k;
  *h = s.h0 + i - k * a.hpk;
}

// Whether a block's output goes straight to the caller's tensors.
__device__ __forceinline__ bool chunk_whole(const ChunkSegment &s) { return s.more == 0; }

// A bf16 pair with a value that is not finite.
__device__ __forceinline__ bool odd_pair(uint32_t w) {
  return (w & 0x7F80u) == 0x7F80u || (w & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ bool odd8(const uint4 &v) {
  return odd_pair(v.x) | odd_pair(v.y) | odd_pair(v.z) | odd_pair(v.w);
}

// Whether V of tokens that are multiplied for the block, but not seen by all of its rows, holds a value
// that is not finite: its new tokens behind the first and what follows in its last tile, and those that
// the window leaves behind between its first row and its last. By `warps` whole warps, each its share
// of 32 tokens at a time: a lane to a token's slot, then a lane to 16 bytes.
__device__ __forceinline__ bool chunk_odd(const ChunkArgs &a, const ChunkSegment &s, int warp,
                                          int warps) {
  const DevLayout &lay = a.lay;
  const bool gqa = lay.kind == KAMERA_GQA;
  const int lane = threadIdx.x & 31;
  const int row = gqa ? lay.row_v : lay.row_k;
  const __nv_bfloat16 *v = (gqa ? a.pool.v : a.pool.k) +
                           (long long)a.layer * a.pool.num_slots * row + (gqa ? s.kvh * lay.hd : 0) +
                           s.part * a.shape.vw;
  const int pieces = min(a.shape.vw, a.dv - s.part * a.shape.vw) >> 3;  // of 16 bytes
  const int sh = a.shape.tile_sh, end = (((s.first + s.ntok - 1) >> sh) + 1) << sh;
  bool odd = false;
  auto slot_at = [&](int t, int to) {
    if (t + lane >= to) return -1;
    const int page = load_page(a, s.r, t + lane);
    if (page < 0 || ((long long)page + 1) * lay.page_size > a.pool.num_slots) return -1;
    return page * lay.page_size + (t + lane - page_index(a, t + lane) * lay.page_size);
  };
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    const int from = side ? first_seen(a, s.first) : s.first + 1;
    const int to = side ? first_seen(a, s.first + s.ntok - 1) : min(s.ctx, end);
    int next = slot_at(from + 32 * warp, to);
#pragma unroll 1
    for (int t = from + 32 * warp; t < to; t += 32 * warps) {
      const int slot = next;
      next = slot_at(t + 32 * warps, to);  // ahead of its use
      const int count = min(32, to - t) * pieces;
#pragma unroll 1
      for (int e0 = 0; e0 < count; e0 += 256) {
        uint4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int e = e0 + 32 * k + lane, i = e / pieces;
          const int at = __shfl_sync(0xffffffffu, slot, min(i, 31));
          x[k] = e < count && at >= 0 ? __ldg(reinterpret_cast<const uint4 *>(
                                                  v + (long long)at * row) + (e - i * pieces))
                                      : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) odd |= odd8(x[k]);
      }
    }
  }
  return odd;
}

// The record of a worker.
__device__ __forceinline__ void chunk_note(ChunkRecord *rec, const ChunkSegment &last, int segments,
                                           bool gave_up, bool odd) {
  ChunkRecord c;
  c.head = segments > 0 && last.more > 0;
  c.more = last.more;
  c.row = last.row;
  c.rows = last.ntok * last.heads;
  c.h0 = last.h0;
  c.part = last.part;
  c.gave_up = gave_up;
  c.odd = odd;
  *rec = c;
}

}  // namespace kamera
