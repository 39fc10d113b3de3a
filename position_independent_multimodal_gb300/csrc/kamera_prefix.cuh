// Work division of attention over shared prefixes, used by its plan, attention and merge
// kernels.
//
// A block is a set of query rows that read the same KV head and the same tokens: (request, query
// head) rows of a group for the group's prefix, or one request's rows for the tokens after it.
// Blocks come in two classes, each with an attention kernel of its own: wide ones (more rows
// than `wide_rows`, tcgen05 tiles of 128 rows) and thin ones (few rows: the bytes of K and V
// bound them, and a tile of 128 rows would be idle for the most part). A unit is one tile of
// tokens (at multiples of the class's tile) of one block of at most `rb` rows. A class's units
// are numbered prefix blocks first (group, KV head and column half, row block, tile), then own
// blocks (request, ...). Workers take consecutive units, as many as one another: every one has the
// same number of tiles whatever the lengths, and cuts at most its first and last block. Where there
// are wide blocks of prefixes alone and workers enough, each block is shared out among workers of
// its own instead, so that no worker has parts of two blocks and those of the blocks of one KV head
// read the same tokens at the same time. A block's first segment writes its rows' partial output to
// the rows' home place, with the number of workers that follow on the block; those write to their
// carry places. The merge kernel joins a row's parts by their log-sum-exp.
#pragma once

#include "kamera_dev.cuh"

namespace kamera {

// What the plan kernel leaves for the others, in the workspace.
struct PrefixPlan {
  // per class c at head[8 c + .]: 0 units U, 1 groups listed, 2 U / n and 3 U % n for the n workers
  // with units, 4 n, 7 units of prefixes. head[16]: requests listed
  long long *head;
  int *gave_up;           // 0 by the plan, 1 by a wide CTA that gave up
  struct Lists {          // blocks of a class
    long long *g_u0;      // [R] first unit of the i-th listed group
    int *g_first, *g_size, *g_prefix, *g_lead;  // first request, requests, prefix, leader
    int4 *start;          // [n][3] the wide class: each worker's first block: list index (own:
                          //     + 2^30), row block, KV head x half, tile; the listed entry's first
                          //     request, requests, leader, first token; end of its tokens, and if
                          //     the block has workers of its own this one's tiles and how many
                          //     workers follow, else -, -1
    float *carry_lse;     // [n][rb]
    float *carry_o;       // [n][rb][dv / vh]
  } cls[2];
  long long *r_u0;        // [R] first own unit of the i-th listed request
  int *r_list;            // [R] listed requests
  int *r_from, *r_to;     // [R] of each: first own token and the end of its context
  long long *gr_u0;       // [R] group g: first unit of its prefix, -1 without one
  int *lead;              // [R] group g: first request with tokens
  long long *req_pu0;     // [R] request r: first unit of its group's prefix, -1 without one
  long long *req_ou0;     // [R] request r: first own unit, -1 without own tokens
  int *req_state;         // [R] 0: outputs not written, 1: written
  int *req_group;         // [R] request r: its group, -1 when it has no tokens
  int *req_at, *req_size; // [R] request r: its place in its group, requests of the group
  int *req_prefix;        // [R] request r: tokens of its group's prefix
  float *home_lse;        // [2][2][R][hq]: prefix and own part, column half
  int2 *home_more;        // [2][2][R][hq]: of the row's first carry place its index in carry_lse,
                          // and how many carries follow (each rb further on)
  float *home_o;          // [2][R][hq][dv]
  size_t total;
};

__host__ __device__ inline PrefixPlan prefix_plan(const PrefixShape &sh, void *ws, long long R,
                                                  int hq, int dv) {
  PrefixPlan p;
  // partial outputs are written by whole lines of 128 bytes
  const size_t skew = static_cast<size_t>(-reinterpret_cast<intptr_t>(ws)) & 127;
  unsigned char *b = static_cast<unsigned char *>(ws) + skew;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    unsigned char *at = b + o;
    o += (bytes + 127) & ~static_cast<size_t>(127);
    return at;
  };
  auto i64 = [&]() { return reinterpret_cast<long long *>(take(8 * R)); };
  auto i32 = [&](long long n) { return reinterpret_cast<int *>(take(4 * n)); };
  auto f32 = [&](long long n) { return reinterpret_cast<float *>(take(4 * n)); };
  p.head = reinterpret_cast<long long *>(take(256));
  p.gave_up = reinterpret_cast<int *>(p.head + 17);
  for (int c = 0; c < 2; ++c) {
    const PrefixClass &k = sh.cls[c];
    p.cls[c].g_u0 = i64();
    p.cls[c].g_first = i32(R);
    p.cls[c].g_size = i32(R);
    p.cls[c].g_prefix = i32(R);
    p.cls[c].g_lead = i32(R);
    p.cls[c].start = reinterpret_cast<int4 *>(take(c == 0 ? 48ll * k.n : 0));
    p.cls[c].carry_lse = f32((long long)k.n * k.rb);
    p.cls[c].carry_o = f32((long long)k.n * k.rb * (dv / k.vh));
  }
  p.r_u0 = i64();
  p.gr_u0 = i64();
  p.req_pu0 = i64();
  p.req_ou0 = i64();
  p.r_list = i32(R);
  p.r_from = i32(R);
  p.r_to = i32(R);
  p.lead = i32(R);
  p.req_state = i32(R);
  p.req_group = i32(R);
  p.req_at = i32(R);
  p.req_size = i32(R);
  p.req_prefix = i32(R);
  p.home_lse = f32(4 * R * hq);
  p.home_more = reinterpret_cast<int2 *>(take(32 * R * hq));
  p.home_o = f32(2 * R * hq * dv);
  p.total = o + 112;  // the workspace is 16-byte aligned
  return p;
}

__host__ __device__ inline int ceil_div(int a, int b) { return (int)(((unsigned)a + b - 1) / b); }

// Tiles of 2^sh tokens that tokens [from, to) lie in.
__host__ __device__ inline int tiles_of(int from, int to, int sh) {
  return to > from ? (int)(((unsigned)to + (1u << sh) - 1) >> sh) - (from >> sh) : 0;
}

// The class of a block with that many rows.
__host__ __device__ inline int class_of(const PrefixShape &sh, int rows) {
  return rows > sh.wide_rows ? 0 : 1;
}

// First unit of worker w.
__device__ __forceinline__ long long first_unit(long long quot, long long rem, long long w) {
  return w * quot + (w < rem ? w : rem);
}
__device__ __forceinline__ long long div_pos(long long a, long long b) {  // a >= 0, b > 0
  if (((a | b) >> 32) == 0) return (unsigned)a / (unsigned)b;
  return a / b;
}
// Workers from w on that take `units` units, the last of them perhaps in part.
__device__ __forceinline__ int workers_for(long long quot, long long rem, long long w,
                                           long long units) {
  const long long n = rem > w ? rem - w : 0, edge = n * (quot + 1);  // those with one unit more
  return (int)(units <= edge ? div_pos(units + quot, quot + 1)
                             : n + div_pos(units - edge + quot - 1, quot));
}

// A run of tiles of one block, as a worker takes it.
struct Segment {
  int own;          // 0: a group's prefix, 1: a request's own tokens
  int r0;           // first request of the rows (own: the request)
  int lead;         // page-table row the tokens are read through
  int row0, rows;   // rows of the block: first (request, head) index in (group x heads), count
  int kvh, half;    // KV head, column half of V
  int tok0, tok1;   // tokens [tok0, tok1) of the segment
  int carry;        // 1: starts inside its block
  int more;         // first segment of its block: how many workers follow on the block
};

// Walks the segments of a worker of class C.
template <int C>
struct SegmentWalk {
  long long u, end;          // units left: [u, end)
  int i, own;                // list index, which list
  int first, size, lead, from, to;  // the listed group or request
  int tiles, nrb;            // tiles and row blocks of each of its blocks
  int rbk, kh, t;            // the next block (row block, KV head x half) and tile
  int worker, groups;        // groups: of the class's list
  int follow;                // the block has workers of its own: those after this one; else -1
  long long quot, rem;       // U / n and U % n

  __device__ __forceinline__ void entry(const PrefixArgs &a, const PrefixPlan &p) {
    if (own) {
      first = lead = p.r_list[i];
      size = 1;
      from = p.r_from[i];
      to = p.r_to[i];
    } else {
      first = p.cls[C].g_first[i];
      size = p.cls[C].g_size[i];
      lead = p.cls[C].g_lead[i];
      from = 0;
      to = p.cls[C].g_prefix[i];
    }
    count(a);
  }
  __device__ __forceinline__ void count(const PrefixArgs &a) {
    tiles = tiles_of(from, to, a.shape.cls[C].tile_sh);
    nrb = ceil_div(size * a.hpk, a.shape.cls[C].rb);
  }
  // By whole warps. Wide: one round of loads; the place is there for every worker, whether or not
  // it has units. Thin: a search by the warp; the plan would take 0.7 us for each 256 workers.
  __device__ __forceinline__ void start(const PrefixArgs &a, const PrefixPlan &p, int worker_) {
    const long long *head = p.head + 8 * C;
    int4 at, e, last;
    if (C == 0) {
      const int4 *rec = p.cls[C].start + 3 * worker_;
      at = rec[0];
      e = rec[1];
      last = rec[2];
    }
    const long long n = head[4], own0 = head[7];
    const int requests = (int)p.head[16];
    worker = worker_;
    groups = (int)head[1];
    quot = head[2];
    rem = head[3];
    u = end = 0;
    follow = -1;
    if (worker >= n) return;
    u = first_unit(quot, rem, worker);
    end = first_unit(quot, rem, worker + 1);
    if (C == 1) {
      own = u >= own0;
      const long long *u0 = own ? p.r_u0 : p.cls[C].g_u0;
      const int lane = threadIdx.x & 31;
      long long from_u = 0;
      i = 0;  // the last listed one that starts at or before u
      for (int len = own ? requests : groups; len > 0;) {
        const int step = (len + 31) >> 5, k = i + lane * step;
        const long long v = lane * step < len ? u0[k] : 0x7FFFFFFFFFFFFFFFll;
        const int j = __popc(__ballot_sync(0xffffffffu, v <= u)) - 1;
        from_u = __shfl_sync(0xffffffffu, v, j);
        i += j * step;
        len = step == 1 ? 0 : min(step, len - j * step);
      }
      entry(a, p);
      const long long d = u - from_u, b = div_pos(d, tiles), h = div_pos(b, nrb);
      rbk = (int)(b - h * nrb);
      kh = (int)h;
      t = (int)(d - b * tiles);
      return;
    }
    own = at.x >> 30;
    i = at.x & 0x3FFFFFFF;
    first = e.x;
    size = e.y;
    lead = e.z;
    from = e.w;
    to = last.x;
    if (last.z >= 0) {
      u = 0;
      end = last.y;
      follow = last.z;
    }
    count(a);
    rbk = at.y;
    kh = at.z;
    t = at.w;
  }
  // The next segment; false when there is none.
  __device__ __forceinline__ bool next(const PrefixArgs &a, const PrefixPlan &p, Segment *s) {
    if (u >= end) return false;
    const PrefixClass &k = a.shape.cls[C];
    if (kh == a.n_kv * k.vh) {  // the entry is done
      ++i;
      if (!own && i == groups) {
        own = 1;
        i = 0;
      }
      entry(a, p);
      kh = 0;
    }
    s->own = own;
    s->r0 = first;
    s->lead = lead;
    s->kvh = k.vh == 1 ? kh : kh >> 1;
    s->half = k.vh == 1 ? 0 : kh & 1;
    s->row0 = rbk * k.rb;
    s->rows = min(k.rb, size * a.hpk - s->row0);
    const long long left = end - u;
    const int nt = (int)(left < tiles - t ? left : tiles - t), t0 = from >> k.tile_sh;
    s->tok0 = t == 0 ? from : (t0 + t) << k.tile_sh;
    s->tok1 = t + nt == tiles ? to : (t0 + t + nt) << k.tile_sh;
    s->carry = t > 0;
    s->more = 0;
    if (t == 0 && nt < tiles)
      s->more = follow >= 0 ? follow : workers_for(quot, rem, worker + 1, tiles - nt);
    u += nt;
    t = 0;
    if (++rbk == nrb) {
      rbk = 0;
      ++kh;
    }
    return true;
  }
};

// (request, query head) of row i of a segment's block. k / hpk by a product: k < 2^24 and
// magic = ceil(2^40 / hpk) is exact for k < 2^40 / hpk^2.
__device__ __forceinline__ void segment_row(const PrefixArgs &a, const Segment &s, int i, int *r,
                                            int *h) {
  const int k = s.row0 + i;
  const int d = (int)((unsigned long long)k * a.hpk_magic >> 40);
  *r = s.r0 + d;
  *h = s.kvh * a.hpk + (k - d * a.hpk);
}

// Where row i of the segment of a worker goes: its output row (dv / vh columns) and its lse. A
// home place also gets what follows on it.
template <int C>
__device__ __forceinline__ void segment_out(const PrefixArgs &a, const PrefixPlan &p,
                                            const Segment &s, int worker, int i, bool tell,
                                            float **o, float **lse) {
  const PrefixClass &c = a.shape.cls[C];
  const int dvh = a.dv / c.vh;
  if (s.carry) {
    const long long k = (long long)worker * c.rb + i;
    *o = p.cls[C].carry_o + k * dvh;
    *lse = p.cls[C].carry_lse + k;
    return;
  }
  int r, h;
  segment_row(a, s, i, &r, &h);
  const long long rh = (long long)r * a.hq + h, n = (long long)a.n_reqs * a.hq;
  const long long z = ((long long)s.own * 2 + s.half) * n + rh;
  *o = p.home_o + (s.own * n + rh) * a.dv + s.half * dvh;
  *lse = p.home_lse + z;
  if (tell) p.home_more[z] = make_int2((worker + 1) * c.rb + i, s.more);
}

// Logical token tok's index in the page table and within its page.
__device__ __forceinline__ int page_index(const PrefixArgs &a, int tok) {
  return a.page_shift >= 0 ? tok >> a.page_shift
                           : (int)((unsigned)tok / (unsigned)a.lay.page_size);
}
// A page-table entry as loaded, before its check. Read-only loads: the plan kernel does not start
// early, so whatever wrote the table was complete before any kernel of the call.
__device__ __forceinline__ int load_page(const PrefixArgs &a, int lead, int tok) {
  return __ldg(a.pool.pt + (long long)lead * a.pool.pt_stride + page_index(a, tok));
}
// Its token's slot; -1 (and the OOB bit) when the page ends outside the pool.
__device__ __forceinline__ int slot_in(const PrefixArgs &a, int page, int tok) {
  const int ps = a.lay.page_size;
  if (page < 0 || ((long long)page + 1) * ps > a.pool.num_slots) {
    atomicOr(a.status, KAMERA_DEVICE_SLOT_OOB);
    return -1;
  }
  return page * ps + (tok - page_index(a, tok) * ps);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two float32 rounded to a pair of bf16, lo in the low half.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

}  // namespace kamera
