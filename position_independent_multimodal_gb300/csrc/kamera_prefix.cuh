// Work division of attention over shared prefixes, used by its plan, attention and merge
// kernels.
//
// A block is a set of query rows that read the same KV head and the same tokens: up to `rb`
// (request, query head) rows of a group for the group's prefix, or one request's rows for the
// tokens after it. A unit is one tile of `tile` tokens of one block; units are numbered prefix
// blocks first (group, KV head and column half, row block, tile), then own blocks (request, ...).
// Tiles lie at multiples of `tile` tokens, so a request's own part starts and ends inside one.
// CTA c of n takes units [c U / n, (c + 1) U / n), so every CTA has the same number of tiles
// whatever the lengths; a range cuts at most its first and last block. A block's first segment
// writes its rows' partial output to the rows' home place, a segment that starts inside a block
// to its CTA's carry place, and the merge kernel adds up a row's parts by their log-sum-exp.
#pragma once

#include "kamera_dev.cuh"

namespace kamera {

// What the plan kernel leaves for the others, in the workspace.
struct PrefixPlan {
  long long *head;      // [0] units, [1] groups with a prefix, [2] requests with own tokens,
                        // [3] CTAs with units, [4] units of the prefixes
  long long *g_u0;      // [R] first unit of the i-th listed group
  long long *r_u0;      // [R] first unit of the i-th listed request
  long long *req_pu0;   // [R] request r: first unit of its group's prefix, -1 without one
  long long *req_ou0;   // [R] request r: first own unit, -1 without own tokens
  int *g_list;          // [R] listed groups: first request, requests, prefix, leader
  int *g_size, *g_prefix, *g_lead;
  int *r_list;          // [R] listed requests
  int *r_from;          // [R] of each listed request: first own token
  int *r_to;            //     and the end of its context
  long long *gr_u0;     // [R] group g: first unit of its prefix, -1 without one
  int *lead;            // [R] group g: first request with tokens
  int *req_state;       // [R] 0: outputs not written, 1: written
  int *req_group;       // [R] request r: its group, -1 when it has no tokens
  int *req_at;          // [R] request r: its place in its group
  int *req_size;        // [R] request r: requests of its group
  int *req_tiles;       // [R] request r: tiles of its group's prefix
  int *req_own;         // [R] request r: tiles of its own tokens
  float *home_lse;      // [2][vh][R][hq]
  float *carry_lse;     // [n][rb]
  float *home_o;        // [2][R][hq][dv]
  float *carry_o;       // [n][rb][dv / vh]
  size_t total;
};

__host__ __device__ inline PrefixPlan prefix_plan(void *ws, long long R, int hq, int dv, int vh,
                                                  int rb, int n) {
  PrefixPlan p;
  unsigned char *b = static_cast<unsigned char *>(ws);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    unsigned char *at = b + o;
    o += (bytes + 15) & ~static_cast<size_t>(15);
    return at;
  };
  auto i64 = [&]() { return reinterpret_cast<long long *>(take(8 * R)); };
  auto i32 = [&]() { return reinterpret_cast<int *>(take(4 * R)); };
  p.head = reinterpret_cast<long long *>(take(64));
  p.g_u0 = i64();
  p.r_u0 = i64();
  p.req_pu0 = i64();
  p.req_ou0 = i64();
  p.gr_u0 = i64();
  p.lead = i32();
  p.g_list = i32();
  p.g_size = i32();
  p.g_prefix = i32();
  p.g_lead = i32();
  p.r_list = i32();
  p.r_from = i32();
  p.r_to = i32();
  p.req_state = i32();
  p.req_group = i32();
  p.req_at = i32();
  p.req_size = i32();
  p.req_tiles = i32();
  p.req_own = i32();
  p.home_lse = reinterpret_cast<float *>(take((size_t)8 * vh * R * hq));
  p.carry_lse = reinterpret_cast<float *>(take((size_t)4 * n * rb));
  p.home_o = reinterpret_cast<float *>(take((size_t)8 * R * hq * dv));
  p.carry_o = reinterpret_cast<float *>(take((size_t)4 * n * rb * (dv / vh)));
  p.total = o;
  return p;
}

__host__ __device__ inline int ceil_div(int a, int b) { return (int)(((unsigned)a + b - 1) / b); }

// Tiles that tokens [from, to) lie in.
__host__ __device__ inline int tiles_of(int from, int to, int tile) {
  return to > from ? ceil_div(to, tile) - from / tile : 0;
}

// A run of tiles of one block, as an attention CTA takes it.
struct Segment {
  int own;          // 0: a group's prefix, 1: a request's own tokens
  int r0;           // first request of the rows (own: the request)
  int lead;         // page-table row the tokens are read through
  int row0, rows;   // rows of the block: first (request, head) index in (group x heads), count
  int kvh, half;    // KV head, column half of V
  int tok0, tok1;   // tokens [tok0, tok1) of the segment
  int carry;        // 1: starts inside its block
};

// Walks the segments of units [u, end).
struct SegmentWalk {
  long long u, end;
  int i;            // index in the group or request list
  __device__ __forceinline__ void start(const PrefixArgs &a, const PrefixPlan &p, int c) {
    const long long U = p.head[0], n = p.head[3];
    u = end = 0;
    i = 0;
    if (c >= n) return;
    // U < 2^62 / n: at most 2^31 requests' tiles
    u = U * c / n;
    end = U * (c + 1) / n;
    const bool own = u >= p.head[4];
    const long long *u0 = own ? p.r_u0 : p.g_u0;
    int lo = 0, hi = (int)(own ? p.head[2] : p.head[1]) - 1;
    while (lo < hi) {  // the last listed one that starts at or before u
      const int mid = (lo + hi + 1) >> 1;
      if (u0[mid] <= u)
        lo = mid;
      else
        hi = mid - 1;
    }
    i = lo;
  }
  // The next segment; false when there is none.
  __device__ __forceinline__ bool next(const PrefixArgs &a, const PrefixPlan &p, Segment *s) {
    if (u >= end) return false;
    const bool own = u >= p.head[4];
    const int n_kv = a.n_kv, hpk = a.hq / n_kv;
    int rows_all, tiles, from, to;
    long long base;
    if (own) {
      if (u == p.head[4]) i = 0;
      if (i + 1 < (int)p.head[2] && u >= p.r_u0[i + 1]) ++i;
      base = p.r_u0[i];
      s->r0 = s->lead = p.r_list[i];
      from = p.r_from[i];
      to = p.r_to[i];
      rows_all = hpk;
    } else {
      if (i + 1 < (int)p.head[1] && u >= p.g_u0[i + 1]) ++i;
      base = p.g_u0[i];
      s->r0 = p.g_list[i];
      s->lead = p.g_lead[i];
      from = 0;
      to = p.g_prefix[i];
      rows_all = p.g_size[i] * hpk;
    }
    tiles = tiles_of(from, to, a.tile);
    const int nrb = ceil_div(rows_all, a.rb);
    const long long b = (u - base) / tiles;  // block: (KV head, half, row block)
    const int t = (int)(u - base - b * tiles);
    const long long kh = b / nrb;
    const int rbk = (int)(b - kh * nrb);
    s->own = own;
    s->kvh = (int)(kh / a.vh);
    s->half = (int)(kh - (long long)s->kvh * a.vh);
    s->row0 = rbk * a.rb;
    s->rows = min(a.rb, rows_all - s->row0);
    const long long left = end - u;
    const int nt = (int)(left < tiles - t ? left : tiles - t);
    s->tok0 = t == 0 ? from : (from / a.tile + t) * a.tile;
    s->tok1 = t + nt == tiles ? to : (from / a.tile + t + nt) * a.tile;
    s->carry = t > 0;
    u += nt;
    return true;
  }
};

// (request, query head) of row i of a segment's block.
__device__ __forceinline__ void segment_row(const PrefixArgs &a, const Segment &s, int i, int *r,
                                            int *h) {
  const int hpk = a.hq / a.n_kv, k = s.row0 + i;
  const int d = k / hpk;
  *r = s.r0 + d;
  *h = s.kvh * hpk + (k - d * hpk);
}

// Where row i of the segment of CTA c goes: its output row (dv / vh columns) and its lse.
__device__ __forceinline__ void segment_out(const PrefixArgs &a, const PrefixPlan &p,
                                            const Segment &s, int c, int i, float **o,
                                            float **lse) {
  const int dvh = a.dv / a.vh;
  if (s.carry) {
    const long long k = (long long)c * a.rb + i;
    *o = p.carry_o + k * dvh;
    *lse = p.carry_lse + k;
    return;
  }
  int r, h;
  segment_row(a, s, i, &r, &h);
  const long long rh = (long long)r * a.hq + h, n = (long long)a.n_reqs * a.hq;
  *o = p.home_o + (s.own * n + rh) * a.dv + s.half * dvh;
  *lse = p.home_lse + ((long long)s.own * a.vh + s.half) * n + rh;
}

}  // namespace kamera
