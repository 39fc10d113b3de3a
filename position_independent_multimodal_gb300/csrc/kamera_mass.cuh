// Work division of the attention masses, used by its kernels. The batch is that of attention over
// chunks of new tokens (kamera_chunk.cuh).
//
// A block is a tile of kt cached tokens of a request; its units are the tiles of new tokens that
// see one of them (tb consecutive ones with the query heads of one KV head, at most qr rows), KV
// head by KV head. Units are numbered by request, tile of cached tokens, KV head, tile of new
// tokens; workers take consecutive ones, as many as one another. So all that is laid on a token is
// added up by one worker, in a fixed order, and each worker cuts at most its first and last block:
// of a cut block every worker leaves its sums, and the join kernel adds them in the workers' order.
#pragma once

#include "kamera_chunk.cuh"

namespace kamera {

struct MassRecord {
  int head;          // 1: its last segment is the first part of a cut block
  int more;          // of that block: workers that follow on it
  int r, tok0;       // of it: request, first token
  int gave_up;
  int pad[3];
};

struct MassPlaces {
  MassRecord *rec;   // [n]
  float *sum;        // [n][2][kt]: carry, home
  size_t total;
};

__host__ __device__ inline MassPlaces mass_places(const MassShape &s, void *ws) {
  MassPlaces p;
  const size_t skew = static_cast<size_t>(-reinterpret_cast<intptr_t>(ws)) & 127;
  unsigned char *b = static_cast<unsigned char *>(ws) + skew;
  const size_t rec = (sizeof(MassRecord) * s.n + 127) & ~static_cast<size_t>(127);
  p.rec = reinterpret_cast<MassRecord *>(b);
  p.sum = reinterpret_cast<float *>(b + rec);
  p.total = rec + 8ull * s.n * s.kt + 112;  // the workspace is 16-byte aligned
  return p;
}

// First and last (exclusive) tile of a request's cached tokens that new tokens see.
__device__ __forceinline__ int mass_tile0(const MassArgs &a, const ChunkRequest &q) {
  return first_seen(a.b, q.past) / a.shape.kt;
}
__device__ __forceinline__ int mass_tiles(const MassArgs &a, const ChunkRequest &q) {
  return ceil_div(q.ctx, a.shape.kt);
}

// Tiles of new tokens that see tokens of tile j: [*i0, *i1).
__device__ __forceinline__ void mass_seen(const MassArgs &a, const ChunkRequest &q, int j, int *i0,
                                          int *i1) {
  const int tok = j * a.shape.kt;
  *i0 = tok > q.past ? (tok - q.past) / a.b.tb : 0;
  const long long lim = (long long)tok + a.shape.kt + a.b.window - 1 - q.past;
  *i1 = a.b.window > 0 && lim < q.n ? ceil_div((int)lim, a.b.tb) : q.nb;
}

// Units of a request's tiles [j0, j) for one KV head, j0 its first.
__device__ __forceinline__ long long mass_units(const MassArgs &a, const ChunkRequest &q, int j0,
                                                int j) {
  const int kt = a.shape.kt, tb = a.b.tb;
  long long sum;
  if (a.b.window == 0) {
    sum = (long long)(j - j0) * q.nb;
  } else {
    // tiles before jx are not seen by the last new tokens
    const long long over = (long long)q.n + q.past - (a.b.window - 1);
    const int jx = over > 0 ? max(j0, (int)((over + kt - 1) / kt) - 1) : j0;
    const int k = min(j, jx) - j0;
    sum = (long long)(j - j0 - k) * q.nb;
    if (k > 0)
      sum += floor_sum(k, tb, kt, (unsigned)((j0 + 1) * kt + a.b.window - 1 - q.past + tb - 1));
  }
  const int x = max(q.past / kt + 1, j0);  // tiles from x on are not seen by the first ones
  if (j > x) sum -= floor_sum(j - x, tb, kt, (unsigned)(x * kt - q.past));
  return sum;
}

// Where a worker starts, found by all threads of the CTA, as chunk_start.
template <int THR>
__device__ __forceinline__ ChunkStart mass_start(const MassArgs &a, int worker,
                                                 ChunkScratch<THR> *sh) {
  return units_start<THR>(a.b, a.shape.n, 1, worker, sh, [&](const ChunkRequest &q) {
    return (long long)a.b.n_kv * a.b.pieces *
           mass_units(a, q, mass_tile0(a, q), mass_tiles(a, q));
  });
}

// Units [k0, k1) of one block.
struct MassSegment {
  ChunkRequest q;
  int r, tok0;      // the request, the block's first token
  int i0, ni;       // its tiles of new tokens
  int k0, k1;
  int carry, more;
};

struct MassWalk {
  ChunkRequest q;
  long long left, quot, rem;
  int r, j, k, worker;  // the next block and its next unit

  __device__ __forceinline__ void start(const MassArgs &a, const ChunkStart &s, int worker_) {
    worker = worker_;
    left = s.units;
    quot = s.quot;
    rem = s.rem;
    r = s.r;
    if (left == 0) return;
    bool bs, bi;
    q = chunk_request(a.b, r, &bs, &bi);
    const int lane = threadIdx.x & 31, heads = a.b.n_kv * a.b.pieces, j0 = mass_tile0(a, q);
    j = j0;  // the last block that starts at or before the unit
    for (int len = mass_tiles(a, q) - j0; len > 1;) {
      const int step = (len + 31) >> 5, at = j + lane * step;
      const bool in =
          lane * step < len && (lane == 0 || heads * mass_units(a, q, j0, at) <= s.off);
      const int i = __popc(__ballot_sync(0xffffffffu, in)) - 1;
      j += i * step;
      len = step == 1 ? 1 : min(step, len - i * step);
    }
    k = (int)(s.off - heads * mass_units(a, q, j0, j));
  }
  __device__ __forceinline__ bool next(const MassArgs &a, MassSegment *s) {
    if (left == 0) return false;
    if (j == mass_tiles(a, q)) {
      do {
        bool bs, bi;
        q = chunk_request(a.b, ++r, &bs, &bi);
      } while (q.n == 0);
      j = mass_tile0(a, q);
      k = 0;
    }
    int i1;
    mass_seen(a, q, j, &s->i0, &i1);
    s->ni = i1 - s->i0;
    s->q = q;
    s->r = r;
    s->tok0 = j * a.shape.kt;
    const int units = a.b.n_kv * a.b.pieces * s->ni;
    const int take = (int)(left < units - k ? left : units - k);
    s->k0 = k;
    s->k1 = k + take;
    s->carry = k > 0;
    s->more = k == 0 && take < units ? workers_for(quot, rem, worker + 1, units - take) : 0;
    left -= take;
    k = 0;
    ++j;
    return true;
  }
};

// Where the sum of token i of a block goes that `worker` has whole, or its part of a cut one.
__device__ __forceinline__ void mass_out(const MassArgs &a, const MassPlaces &p,
                                         const MassSegment &s, int worker, int i, float sum) {
  if (s.carry || s.more) {
    p.sum[(2ll * worker + (s.carry ? 0 : 1)) * a.shape.kt + i] = sum;
  } else if (s.tok0 + i < s.q.ctx) {
    float *m = a.mass + (long long)s.r * a.mass_stride + s.tok0 + i;
    *m = a.decay == 0.f ? sum : fmaf(a.decay, *m, sum);
  }
}

__device__ __forceinline__ void mass_note(MassRecord *rec, const MassSegment &last, int segments,
                                          bool gave_up) {
  MassRecord c;
  c.head = segments > 0 && last.more > 0;
  c.more = last.more;
  c.r = last.r;
  c.tok0 = last.tok0;
  c.gave_up = gave_up;
  *rec = c;
}

}  // namespace kamera
