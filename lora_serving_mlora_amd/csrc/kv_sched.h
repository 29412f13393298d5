// How the attention's work is dealt to a fixed number of workgroups when the
// lengths are only known on the device.
//
// An item is a tile of R rows of one (sequence, key/value head); it walks its
// visible tokens in steps of 64.  Items lie on a line in the order (sequence,
// head, tile), each as long as its steps plus `over` for what an item costs
// besides; workgroup w takes the w-th of 2^lw (nearly) equal parts of the
// line, so one long sequence is cut into many pieces and many short ones are
// packed together, and no length is ever read by the host.  A cut that falls
// within 6 steps of an item's end is moved there (by both neighbours alike),
// which keeps pieces from being tiny; farther moves leave long parts unequal
// (an eighth of the part: 256 requests 449 us, not 431; a 2048-token chunk 719
// us, not 654).  The order and the cuts depend on the batch alone, so results
// are the same from call to call.
//
// A cut item's pieces go to the caller's work buffer as (O, M, L) and are
// joined by join_part: worker w's slot 2w holds the piece that its part
// begins inside of, slot 2w + 1 the piece that its part ends inside of.
#pragma once

#include "kv.h"

namespace mlora {

constexpr int kKvStep = 64;  // tokens of a step

struct KvSched {
  int lw;                  // log2 of the workgroups: parts of the line
  int skew;                // 256ths that the parts of the second half take less, see sched_place
  int tiles;               // where workgroup i takes item i whole: tiles of a (sequence, head) at most
  int over, tol_max, mirror, min_share;
  int min_rows, max_rows;  // sequences with other numbers of rows are left out
};

struct Span {
  int lo, hi;  // tokens lo <= t < hi
};

// What new token j of a sequence sees.  What lies past the table is
// represented by its first token there, which has no page, so that a wrong
// kv_len costs no more than a full table.
__device__ __forceinline__ Span row_span(const KvView& c, const KvAttn& a, const KvSeq& s, int j) {
  Span v{0, max(s.n, 0)};
  if (a.causal) {
    v.hi = max(0, s.n - s.m + j + 1);
    if (a.window > 0) v.lo = max(0, v.hi - a.window);
  }
  const int end = c.width << c.lb;
  if (v.hi > end) v = {min(v.lo, end), end + 1};
  return v;
}

// A tile's rows and steps.  Rows: a (sequence, key/value head) has m * G of
// them, row r being new token r / G and query head h * G + r % G.
template <int R>
struct Tile {
  int r0, r1;          // first and last row
  int lo, hi;          // tokens seen by some row
  int every_lo, every_hi;  // tokens seen by every row
  int step0, steps;    // at least one step

  Tile() = default;
  __device__ __forceinline__ Tile(const KvView& c, const KvAttn& a, const KvSeq& s, int tile) {
    r0 = tile * R;
    r1 = min(r0 + R, s.m * a.G) - 1;
    const Span x = row_span(c, a, s, r0 / a.G), y = row_span(c, a, s, r1 / a.G);
    lo = x.lo;
    hi = y.hi;
    every_lo = y.lo;
    every_hi = x.hi;
    step0 = lo / kKvStep;
    steps = max(1, (hi + kKvStep - 1) / kKvStep - step0);
  }
};

__device__ __forceinline__ bool sched_takes(const KvSched& d, int rows) {
  return rows > d.min_rows && rows <= d.max_rows;
}

// with `mirror` long and short tiles of a causal sequence alternate, so that
// equal parts of the line hold nearly equal numbers of whole items
__device__ __forceinline__ int sched_tile(const KvSched& d, int k, int tiles) {
  return d.mirror ? (k & 1 ? tiles - 1 - (k >> 1) : k >> 1) : k;
}

// a place on the line: `off` into tile number k (in the line's order) of head h
struct SchedPos {
  int64_t p;
  int seq, h, k, off;
};

constexpr int kSchedSeqs = 256;  // sequences whose tiles are dealt with side by side
struct SchedLds {
  int64_t sum[4];
  int64_t cost[kSchedSeqs];  // line length of one head
  int64_t at[2];             // start of the head that holds the place
  SchedPos pos[2];
  int m[kSchedSeqs], n[kSchedSeqs];
  int before[kSchedSeqs + 1];  // tiles of the sequences before
};

// line length of one head of sequence i
template <int R>
__device__ int64_t sched_cost(const KvView& c, const KvAttn& a, const KvSched& d, int i) {
  const KvSeq s = kv_seq(c, i);
  const int rows = s.m * a.G;
  if (!sched_takes(d, rows)) return 0;
  int64_t sum = 0;
  for (int t = 0; t * R < rows; ++t) sum += Tile<R>(c, a, s, t).steps + d.over;
  return sum;
}

template <class T>
__device__ __forceinline__ T wave_scan(T x) {  // inclusive
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int m = 1; m < 64; m <<= 1) {
    const T y = __shfl_up(x, m, 64);
    if (lane >= m) x += y;
  }
  return x;
}

// Where worker w's part begins.  The workgroups of an XCD take neighbouring
// parts; those launched later share their CU with one launched earlier, whose
// waves are served first where both could issue, so each of them takes `skew`
// less and the earlier ones that much more, for both to end together.
__device__ __forceinline__ int64_t sched_place(const KvSched& d, int64_t share, int w) {
  const int per = (1 << d.lw) >> 3, l = w % per, more = l < per / 2 ? l : per - l;
  return share * w + (share * more * d.skew >> 8);
}

// Which head holds the place `off` into a sequence whose heads take `head` each.
// A division in 64 bits takes half a microsecond, so one in 32 serves where
// both fit; one head passes 2^32 for a prompt of 3 M tokens and 8 query heads.
__host__ __device__ __forceinline__ int sched_head(int64_t off, int64_t head) {
  if (off < head) return 0;
  return off <= INT32_MAX ? (int)((uint32_t)off / (uint32_t)head) : (int)(off / head);
}

// The part of worker w: its first place (L.pos[0]) and its end (L.pos[1].p).
// Everything that depends on the number of tiles is done by all 256 threads
// side by side: one thread that went through the tiles of a long prompt alone
// took longer than the products of a short one (8 prompts 90 us, not 66).
template <int R>
__device__ __forceinline__ void sched_part(const KvView& c, const KvAttn& a, const KvSched& d, int w, SchedLds& L) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const bool small = c.n_seq <= kSchedSeqs;
  const int per = (c.n_seq + 255) / 256, i0 = tid * per, i1 = min(i0 + per, c.n_seq);
  int64_t own = 0;
  if (small) {
    int tiles = 0;
    if (tid < c.n_seq) {
      const KvSeq s = kv_seq(c, tid);
      const int rows = s.m * a.G;
      if (sched_takes(d, rows)) tiles = (rows + R - 1) / R;
      L.m[tid] = s.m;
      L.n[tid] = s.n;
    }
    L.cost[tid] = 0;
    int incl = wave_scan(tiles);
    if (lane == 63) L.sum[wave] = incl;
    __syncthreads();
    for (int v = 0; v < wave; ++v) incl += (int)L.sum[v];
    L.before[tid + 1] = incl;
    if (tid == 0) L.before[0] = 0;
    __syncthreads();
    const int all = L.before[kSchedSeqs];
    for (int f = tid; f < all; f += 256) {
      int i = 0;  // the last sequence that begins at or before tile f
#pragma unroll
      for (int x = kSchedSeqs / 2; x > 0; x >>= 1)
        if (L.before[i + x] <= f) i += x;
      const KvSeq s{0, L.m[i], L.n[i]};
      atomicAdd(reinterpret_cast<unsigned long long*>(&L.cost[i]),
                (unsigned long long)(Tile<R>(c, a, s, f - L.before[i]).steps + d.over));
    }
    __syncthreads();
    own = L.cost[tid];
  } else {
    for (int i = i0; i < i1; ++i) own += sched_cost<R>(c, a, d, i);
  }
  own *= c.H;
  int64_t incl = wave_scan(own);
  if (lane == 63) L.sum[wave] = incl;
  __syncthreads();
  int64_t total = 0;
  for (int v = 0; v < 4; ++v) {
    if (v < wave) incl += L.sum[v];
    total += L.sum[v];
  }
  const int64_t share = max<int64_t>((total + (1 << d.lw) - 1) >> d.lw, d.min_share);
  const int64_t tol = min<int64_t>(max<int64_t>(share / 8, d.over), d.tol_max);
  if (tid < 2) L.pos[tid] = {total, -1, 0, 0, 0};  // for ends past the line
  __syncthreads();
  // the sequence and head that hold each place (one thread at most holds it)
#pragma unroll 1
  for (int b = 0; b < 2; ++b) {
    const int64_t p = sched_place(d, share, w + b);
    if (p < incl - own || p >= incl) continue;
    int64_t at = incl - own;
    for (int i = i0; i < i1; ++i) {
      const int64_t head = small ? L.cost[tid] : sched_cost<R>(c, a, d, i);
      if (p >= at + head * c.H) {
        at += head * c.H;
        continue;
      }
      const int h = sched_head(p - at, head);
      L.pos[b] = {p, i, h, 0, 0};
      L.at[b] = at + h * head;
      break;
    }
  }
  __syncthreads();
  // its tile, by a wave for each place
  if (wave < 2 && L.pos[wave].seq >= 0) {
    SchedPos q = L.pos[wave];
    const KvSeq s = kv_seq(c, q.seq);
    const int tiles = (s.m * a.G + R - 1) / R;
    int64_t at = L.at[wave];
    for (int k0 = 0; k0 < tiles; k0 += 64) {
      const int k = k0 + lane;
      const int len = k < tiles ? Tile<R>(c, a, s, sched_tile(d, k, tiles)).steps + d.over : 0;
      const int64_t end = at + wave_scan(len);
      const uint64_t past = __ballot(q.p < end);
      if (past == 0) {
        at = __shfl(end, 63, 64);
        continue;
      }
      if (lane == __builtin_ctzll(past)) {
        const int64_t begin = end - len;
        q.k = k;
        q.off = (int)(q.p - begin);
        if (q.off <= tol) {
          q.off = 0;
          q.p = begin;
        } else if (end - q.p <= tol) {
          q.p = end;
          q.off = len;  // the caller goes on to the next item
        }
        L.pos[wave] = q;
      }
      break;
    }
  }
  __syncthreads();
}

// words of a worker's entry in the work buffer: whether its first piece began
// before its part (0 no, 1 and ends in it, 2 and goes on past it), and the
// item that it begins and does not end (sequence or -1, head, tile)
constexpr int kSchedMeta = 4;
constexpr int kSchedMaxWorkers = 1024;
__host__ __device__ constexpr size_t sched_slot_floats(int R, int D) { return (size_t)R * (D + 2); }
inline size_t sched_bytes(int workers, int R, int D) {
  return (size_t)kSchedMaxWorkers * kSchedMeta * 4 + (size_t)workers * 2 * sched_slot_floats(R, D) * 4;
}
__device__ __forceinline__ int* sched_meta(void* work, int w) { return static_cast<int*>(work) + w * kSchedMeta; }
// slot: O [R][D], M [R], L [R]
__device__ __forceinline__ float* sched_slot(void* work, int slot, int R, int D) {
  return reinterpret_cast<float*>(static_cast<char*>(work) + (size_t)kSchedMaxWorkers * kSchedMeta * 4) +
         (size_t)slot * sched_slot_floats(R, D);
}

// steps s0 <= i < s1 of a tile's, slot < 0 where that is the whole item
template <int R>
struct Piece {
  KvSeq s;
  Tile<R> t;
  int seq, h, tile, s0, s1, slot;
};

// The pieces of this workgroup's part, in their order; the same in every lane.
// WHOLE: no parts, workgroup i takes item i.
template <int R, bool WHOLE>
struct Pieces {
  const KvView& c;
  const KvAttn& a;
  const KvSched& d;
  int64_t left;  // of the part
  int w, first, tail[3], seq, h, k, off;
  KvSeq s;

  __device__ __forceinline__ Pieces(const KvView& c_, const KvAttn& a_, const KvSched& d_, SchedLds& L)
      : c(c_), a(a_), d(d_), left(1), w(blockIdx.x), first(0), tail{-1, 0, 0}, h(0), k(0), off(0) {
    if constexpr (!WHOLE) {
      // neighbours on the line go to one XCD (workgroups are dealt to the 8 in
      // turn), whose L2 then serves the tiles that share keys and values
      w = ((blockIdx.x & 7) << (d.lw - 3)) + (blockIdx.x >> 3);
      sched_part<R>(c, a, d, w, L);
      const SchedPos b = L.pos[0];
      const int64_t length = L.pos[1].p - b.p;
      left = (int64_t)__builtin_amdgcn_readfirstlane((int)(length >> 32)) << 32 |
             (uint32_t)__builtin_amdgcn_readfirstlane((int)length);
      seq = __builtin_amdgcn_readfirstlane(b.seq), h = __builtin_amdgcn_readfirstlane(b.h);
      k = __builtin_amdgcn_readfirstlane(b.k), off = __builtin_amdgcn_readfirstlane(b.off);
      if (left > 0) load();
    }
  }
  __device__ __forceinline__ void load() {
    const KvSeq x = kv_seq(c, seq);
    s.row0 = __builtin_amdgcn_readfirstlane(x.row0);
    s.m = __builtin_amdgcn_readfirstlane(x.m);
    s.n = __builtin_amdgcn_readfirstlane(x.n);
  }

  __device__ __forceinline__ bool next(Piece<R>& p) {
    if constexpr (WHOLE) {
      if (left == 0) return false;
      left = 0;
      // the last tiles, which see most, first; a head's stay on one XCD where
      // there are 8 heads
      int item = blockIdx.x;
      h = item % c.H;
      item /= c.H;
      seq = item % c.n_seq, k = d.tiles - 1 - item / c.n_seq;
      load();
      if (!sched_takes(d, s.m * a.G) || k * R >= s.m * a.G) return false;
      p.t = Tile<R>(c, a, s, k);
      p.s = s, p.seq = seq, p.h = h, p.tile = k, p.s0 = 0, p.s1 = p.t.steps, p.slot = -1;
      return true;
    } else {
      while (left > 0) {
        const int rows = s.m * a.G, tiles = (rows + R - 1) / R;
        if (!sched_takes(d, rows) || h >= c.H) {
          // on to the next sequence that has tiles, 64 looked at together
          h = k = off = 0;
          uint64_t has = 0;
          for (++seq; seq < c.n_seq; seq += 64) {
            const int i = seq + (int)(threadIdx.x & 63);
            has = __ballot(i < c.n_seq && sched_takes(d, kv_seq(c, min(i, c.n_seq - 1)).m * a.G));
            if (has) break;
          }
          if (!has) {
            left = 0;
            break;
          }
          seq += __builtin_ctzll(has);
          load();
          continue;
        }
        if (k >= tiles) {
          k = off = 0;
          ++h;
          continue;
        }
        p.tile = sched_tile(d, k, tiles);
        p.t = Tile<R>(c, a, s, p.tile);
        const int len = p.t.steps + d.over;
        if (off >= len) {
          ++k;
          off = 0;
          continue;
        }
        const int take = (int)min<int64_t>(left, len - off);
        const bool head = off == 0, end = off + take == len;
        if (!head) first = end ? 1 : 2;
        if (head && !end) tail[0] = seq, tail[1] = h, tail[2] = p.tile;
        p.s = s, p.seq = seq, p.h = h;
        p.s0 = max(0, off - d.over), p.s1 = max(0, off + take - d.over);
        p.slot = head && end ? -1 : 2 * w + (head ? 1 : 0);
        left -= take;
        off = 0;
        ++k;
        return true;
      }
      return false;
    }
  }

  // after the last piece: what the join has to know
  __device__ __forceinline__ void finish() {
    if constexpr (!WHOLE) {
      if (threadIdx.x == 0) {
        int* m = sched_meta(a.work, w);
        m[0] = first;
        m[1] = tail[0];
        m[2] = tail[1];
        m[3] = tail[2];
      }
    }
  }
};

// four channels of row rr of a (sequence, head): o / l, zero where the row
// sees nothing (l may also be 0 because every score is -infinity: NaN)
typedef float f32x4 __attribute__((ext_vector_type(4)));
__device__ __forceinline__ bool row_sees(const KvView& c, const KvAttn& a, const KvSeq& s, int rr) {
  const Span x = row_span(c, a, s, rr / a.G);
  return x.hi > x.lo;
}
template <int D>
__device__ __forceinline__ void write_row(const KvAttn& a, const KvSeq& s, int Hq, int h, int rr, int ch, f32x4 o,
                                          float l, bool sees) {
  const float inv = sees ? 1.f / l : 0.f;
  uint16_t* dst = a.out + ((size_t)(s.row0 + rr / a.G) * Hq + h * a.G + rr % a.G) * D + ch;
  *reinterpret_cast<uint2*>(dst) = uint2{pack_bf2_hw(o[0] * inv, o[1] * inv), pack_bf2_hw(o[2] * inv, o[3] * inv)};
}

// Joins the pieces of the item that worker w began and did not end:
// o = sum_i 2^(M_i - M) O_i / sum_i 2^(M_i - M) L_i, the pieces in their order.
// Many pieces (a few rows over a long axis) are read side by side, as one after
// the other they would cost a memory latency each; with few, the rows are.
// blockIdx.y takes a share of the rows.
constexpr int kJoinFew = 8;
template <int R, int D>
__device__ __forceinline__ void join_part(const KvView& c, const KvAttn& a, int workers, int w) {
  constexpr int DL = D / 4, NG = 256 / DL;  // lanes of a row, pieces side by side
  __shared__ __align__(16) float sh[NG][D + 4];
  const int tid = threadIdx.x;
  const int* meta = sched_meta(a.work, w);
  const int seq = meta[1], h = meta[2], tile = meta[3];
  if (seq < 0) return;
  int n = 1;  // the pieces: this one and those of the workers up to the first that ends the item
  for (int w0 = w + 1; w0 < workers; w0 += 64) {
    const int x = w0 + (tid & 63);
    const uint64_t on = __ballot(x < workers && sched_meta(a.work, x)[0] == 2);
    const int run = on == ~0ull ? 64 : __builtin_ctzll(~on);
    n += run;
    if (run < 64) {
      n += (w0 + run < workers);
      break;
    }
  }
  const KvSeq s = kv_seq(c, seq);
  const int r0 = tile * R, cnt = min(R, s.m * a.G - r0), Hq = c.H * a.G;
  const int d = 4 * (tid % DL), grp = tid / DL;
  if (R > 16 || n <= kJoinFew) {
    for (int x = blockIdx.y * 256 + tid; x < cnt * DL; x += gridDim.y * 256) {
      const int r = x / DL, ch = 4 * (x % DL);
      float M = -__builtin_huge_valf(), L = 0.f;
      f32x4 o{0, 0, 0, 0};
      for (int i0 = 0; i0 < n; i0 += kJoinFew) {
        float m[kJoinFew], l[kJoinFew], top = M;
        f32x4 v[kJoinFew];
#pragma unroll
        for (int i = 0; i < kJoinFew; ++i) {
          m[i] = -__builtin_huge_valf();
          l[i] = 0.f;
          v[i] = f32x4{0, 0, 0, 0};
          if (i0 + i < n) {
            const float* slot = sched_slot(a.work, i0 + i == 0 ? 2 * w + 1 : 2 * (w + i0 + i), R, D);
            m[i] = slot[R * D + r], l[i] = slot[R * D + R + r];
            v[i] = *reinterpret_cast<const f32x4*>(slot + r * D + ch);
          }
          top = fmaxf(top, m[i]);
        }
        const float ref = top == -__builtin_huge_valf() ? 0.f : top, f0 = __builtin_amdgcn_exp2f(M - ref);
        M = top;
        L *= f0;
        o *= f0;
#pragma unroll
        for (int i = 0; i < kJoinFew; ++i) {
          const float f = __builtin_amdgcn_exp2f(m[i] - ref);
          L += l[i] * f;
          o += v[i] * f;
        }
      }
      write_row<D>(a, s, Hq, h, r0 + r, ch, o, L, row_sees(c, a, s, r0 + r));
    }
    return;
  }
  for (int r = blockIdx.y; r < cnt; r += gridDim.y) {
    float M = -__builtin_huge_valf(), L = 0.f;
    f32x4 o{0, 0, 0, 0};
    if (grp < NG)
      for (int i = grp; i < n; i += NG) {
        const float* slot = sched_slot(a.work, i == 0 ? 2 * w + 1 : 2 * (w + i), R, D);
        const float m = slot[R * D + r], l = slot[R * D + R + r];
        const f32x4 v = *reinterpret_cast<const f32x4*>(slot + r * D + d);
        const float Mn = fmaxf(M, m), ref = Mn == -__builtin_huge_valf() ? 0.f : Mn;
        const float f = __builtin_amdgcn_exp2f(M - ref), e = __builtin_amdgcn_exp2f(m - ref);
        M = Mn;
        L = L * f + l * e;
        o = o * f + v * e;
      }
    __syncthreads();
    if (grp < NG) {
      *reinterpret_cast<f32x4*>(&sh[grp][d]) = o;
      if (d == 0) sh[grp][D] = M, sh[grp][D + 1] = L;
    }
    __syncthreads();
    if (tid < DL) {
      float top = sh[0][D];
      for (int i = 1; i < NG; ++i) top = fmaxf(top, sh[i][D]);
      const float ref = top == -__builtin_huge_valf() ? 0.f : top;
      float l = 0.f;
      f32x4 v{0, 0, 0, 0};
      for (int i = 0; i < NG; ++i) {
        const float f = __builtin_amdgcn_exp2f(sh[i][D] - ref);
        l += sh[i][D + 1] * f;
        v += *reinterpret_cast<const f32x4*>(&sh[i][d]) * f;
      }
      write_row<D>(a, s, Hq, h, r0 + r, d, v, l, row_sees(c, a, s, r0 + r));
    }
  }
}

}  // namespace mlora
