// Attention over the paged 8-bit key/value cache.
//
// For a row with query q at position x, over the tokens t that it sees:
//   s_t = q . k_t,  p_t = 2^((s_t - M) c),  o = sum_t p_t v_t / sum_t p_t,
// c = scale * log2(e), in one pass: M is a running reference for the largest
// s_t, and what was summed under an older one is multiplied by the quotient.
// The codes become bf16 in registers, times their page's scale: exact, so the
// products lose nothing against an unquantised bf16 cache.  (The 8-bit matrix
// instruction would take the codes as they are and run at twice the rate, but
// it drops what lies 2^-13 below the magnitudes it sums, and the queries
// would need two codes each.)
#include <algorithm>

#include "kv_sched.h"

namespace mlora {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr float kInf = __builtin_huge_valf(), kMax = 0x1.fffffep127f;
constexpr int kWaves = 4;
constexpr float kSlack = 8.f;  // log2 by which a score may pass M before the sums are rescaled

// An exponent is s * cs - ref, one operation.  What ref = M * cs was rounded by,
// 2^-25 of it, is what the exponent of the largest score is off by: too much
// for any probability to stay finite, or above 0, once ref passes 2^31.  From
// kHuge on, scores that differ at all do so by 2^5 in the exponent, so the
// largest has all the weight whatever the factor: a power of two makes ref exact.
constexpr float kHuge = 0x1p30f;
struct Ref {
  float cs, ref;
  __device__ __forceinline__ Ref(float M, float scale) {
    const float pow2 = __uint_as_float(__float_as_uint(scale) & 0x7f800000u);
    cs = fabsf(M * scale) >= kHuge ? pow2 : scale;
    ref = M == -kInf ? 0.f : M * cs;
  }
  __device__ __forceinline__ float p(float s) const { return __builtin_amdgcn_exp2f(__builtin_fmaf(s, cs, -ref)); }
};

__device__ __forceinline__ bf16x8 frag(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, uint4{a, b, c, d});
}
__device__ __forceinline__ bf16x8 frag_fp8(uint32_t lo, uint32_t hi, float s) {
  return frag(kv_bf2<false>(lo, s), kv_bf2<true>(lo, s), kv_bf2<false>(hi, s), kv_bf2<true>(hi, s));
}

// 16 bf16 at p, 16-byte aligned or not
__device__ __forceinline__ void load16(const uint16_t* p, bool vec, uint4& x, uint4& y) {
  if (vec) {
    x = *reinterpret_cast<const uint4*>(p);
    y = *reinterpret_cast<const uint4*>(p + 8);
  } else {
    auto two = [&](int i) { return p[i] | (uint32_t)p[i + 1] << 16; };
    x = uint4{two(0), two(2), two(4), two(6)};
    y = uint4{two(8), two(10), two(12), two(14)};
  }
}

// over the lanes with the same l % 16
__device__ __forceinline__ float max_rows(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(b[0]), __uint_as_float(b[1]));
}
__device__ __forceinline__ float sum_rows(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  x = __uint_as_float(a[0]) + __uint_as_float(a[1]);
  auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(b[0]) + __uint_as_float(b[1]);
}

// bytes of w that are NaN codes, as 0x80 in each
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) { return ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u; }
// 0x80 marks -> ones for each marked byte of the low or high pair, as packed bf16
template <bool HI>
__device__ __forceinline__ uint32_t ones2(uint32_t m) {
  const uint32_t a = HI ? m >> 16 : m;
  return (a & 0x80u ? 0x3f80u : 0u) | (a & 0x8000u ? 0x3f800000u : 0u);
}

// ----------------------------------------------------------------------------
// Few rows: 16 rows of one (sequence, key/value head), four waves that take
// every fourth step of 64 tokens, straight from memory into registers.
//
// One wave's step, S^T = K Q^T and O^T = V^T P^T with 16x16x32 products: lane
// l = 16 g + q holds in S^T's tile t, element e, the score of row q and token
// 16 g + 4 t + e (the keys' rows are dealt to the matrix rows that way), so
// its 16 scores are those of the 16-token block g: exactly the probabilities
// that it has to supply to the second product, whose other operand is the
// block's 16 bytes of a channel, one load.  Nothing passes through LDS.
//
// Bound by reading the cache: 256 requests of 1000 .. 8100 tokens (8 heads of
// 128 channels, 2.4 GB) take 418 us, 5.7 TB/s, where a plain read of 1 GiB
// reaches 6.0; 32 requests of 100 .. 4000 tokens 32 us (3.9 TB/s): the parts
// are found, the first loads arrive, the waves and the pieces are joined, about
// 10 us that no other load hides.
// ----------------------------------------------------------------------------
template <int D>
struct RowsTile {
  static constexpr int R = (D + 63) / 64;  // 16-byte loads of a lane for a token's keys
  static constexpr int T = D / 16;         // channel tiles of the output
  // Workgroups of a CU.  In the form of parts the registers of two hold neither
  // the output nor the next step's loads above 128 channels (256 requests of
  // 1000 .. 8000 tokens: 606 us with one, 790 us with two at 192 channels, 516
  // and 554 us at 160; 64 sequences of 500 .. 4000 at 256: 60 and 99 us).  Whole
  // items, which carry no parts, do better with two up to 192 channels (window
  // of 1024 over 96 sequences: 29.6 us with two, 32.1 us with one; at 160 23.4
  // and 28.8 us).
  static constexpr int PER_CU = D > 128 ? 1 : 2, WHOLE_PER_CU = D > 192 ? 1 : 2;
};

// Loads of the next step are issued as soon as the registers they go to have
// been read (the keys' after the first product, the values' after the second),
// and its page ids a step before that.  An id looked at where it was loaded had
// the wave wait for all loads before it: 256 requests 431 us, not 420.
template <int D>
struct RowsLds {
  float m[kWaves][16], l[kWaves][16];
  float o[kWaves][16][D + 4];
  SchedLds sched;
};

template <int D, bool WHOLE>
__device__ __forceinline__ void rows_part(const KvView& c, const KvAttn& a, const KvSched& d, RowsLds<D>& lds) {
  constexpr int R = RowsTile<D>::R, T = RowsTile<D>::T;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int q = lane & 15, g = lane >> 4, kblk = q >> 2, B = 1 << c.lb;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.q) | (uintptr_t)(a.rs * 2) | (uintptr_t)(a.hs * 2)) & 15u) == 0;
  const float cs = a.scale * 1.4426950408889634f, slack = fminf(kSlack / cs, kMax);

  typedef Piece<16> P;
  bf16x8 qf[R][2];
  auto load_q = [&](const P& p) {
    const int r = min(p.t.r0 + q, p.t.r1), j = r / a.G;
    const uint16_t* src = a.q + (size_t)(p.s.row0 + j) * a.rs + (size_t)(p.h * a.G + r % a.G) * a.hs;
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int u = 4 * i + g;
      uint4 x{}, y{};
      if (16 * u < D) load16(src + 16 * u, vec, x, y);
      qf[i][0] = __builtin_bit_cast(bf16x8, x);
      qf[i][1] = __builtin_bit_cast(bf16x8, y);
    }
  };
  // page ids of this lane's keys (16-token block q / 4 of a step) and values
  // (block g), looked at when they are used: a look here would wait for them,
  // and so for all loads before them
  int kid = 0, vid = 0;
  auto ids = [&](const P& p, int step, int& key, int& value) {
    const int* pages = c.table + (size_t)p.seq * c.table_stride;
    key = pages[min((step * kKvStep + 16 * kblk) >> c.lb, c.width - 1)];
    value = pages[min((step * kKvStep + 16 * g) >> c.lb, c.width - 1)];
  };
  const uint8_t *kptr, *vptr;
  float ks, vs;
  uint4 kw[4][R], vw[T];
  bool bad, vin;
  const float *ksp, *vsp;
  auto place = [&](const P& p, int step) {
    const int kt = step * kKvStep + 16 * kblk, vt = step * kKvStep + 16 * g;
    auto page_at = [&](int id, int tok) {  // -1 where there is none, any for what nobody sees
      if (tok >= p.t.hi) return 0;
      return (tok >> c.lb) < c.width && (unsigned)id < (unsigned)c.n_blocks ? id : -1;
    };
    const int kpage = page_at(kid, kt), vpage = page_at(vid, vt);
    const size_t kp = (size_t)max(kpage, 0) * c.H + p.h, vp = (size_t)max(vpage, 0) * c.H + p.h;
    kptr = c.k + ((kp << c.lb) + (kt & (B - 1)) + (q & 3)) * D;
    vptr = c.v + ((vp << c.lb) + (vt & (B - 1))) * D + q * 16;
    ksp = c.k_scale + kp;
    vsp = c.v_scale + vp;
    bad = vpage < 0;
    vin = !bad && vt < p.t.hi && vt + 16 > p.t.lo;
  };
  auto load_k = [&]() {
    ks = *ksp;
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int i = 0; i < R; ++i) {
        kw[x][i] = uint4{0, 0, 0, 0};
        if (16 * (4 * i + 3) < D || 16 * (4 * i + g) < D)
          kw[x][i] = *reinterpret_cast<const uint4*>(kptr + 4 * x * D + 16 * (4 * i + g));
      }
  };
  auto load_v = [&]() {
    vs = *vsp;
#pragma unroll
    for (int i = 0; i < T; ++i) vw[i] = *reinterpret_cast<const uint4*>(vptr + 256 * i);
  };
  // the loads of a piece's first step, whose ids are here
  auto start = [&](const P& p) {
    const int step = p.t.step0 + p.s0 + wave, end = p.t.step0 + p.s1;
    if (step < end) {
      place(p, step);
      load_k();
      load_v();
      ids(p, step + kWaves, kid, vid);
    }
    load_q(p);
  };

  Pieces<16, WHOLE> pieces(c, a, d, lds.sched);
  P p, next;
  bool have = pieces.next(p);
  if (have) {
    ids(p, p.t.step0 + p.s0 + wave, kid, vid);
    start(p);
  }
  while (have) {
    const Tile<16>& t = p.t;
    const KvSeq& s = p.s;
    const int h = p.h, slot = p.slot;
    const bool have_next = pieces.next(next);
    int next_kid = 0, next_vid = 0;
    if (have_next) ids(next, next.t.step0 + next.s0 + wave, next_kid, next_vid);
    const Span mine = row_span(c, a, s, min(t.r0 + q, t.r1) / a.G);
    f32x4 o[T];
#pragma unroll
    for (int i = 0; i < T; ++i) o[i] = f32x4{0, 0, 0, 0};
    float M = -kInf, L = 0.f;

    const int end = t.step0 + p.s1;
    for (int step = t.step0 + p.s0 + wave; step < end; step += kWaves) {
      const bool more = step + kWaves < end;
      const int base = step * kKvStep;
      const bool bad_now = bad, vin_now = vin;
      f32x4 st[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        st[x] = f32x4{0, 0, 0, 0};
#pragma unroll
        for (int i = 0; i < R; ++i) {
          const bf16x8 lo = frag_fp8(kw[x][i].x, kw[x][i].y, ks), hi = frag_fp8(kw[x][i].z, kw[x][i].w, ks);
          st[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, qf[i][0], st[x], 0, 0, 0);
          st[x] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, qf[i][1], st[x], 0, 0, 0);
        }
      }
      if (more) {
        place(p, step + kWaves);
        load_k();
        ids(p, step + 2 * kWaves, kid, vid);
      }
      const int mt = base + 16 * g;  // first of this lane's 16 tokens
      if (__ballot(bad_now)) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (bad_now) st[x][e] = __builtin_nanf("");
      }
      const float vsc = vin_now ? vs : 1.f;
      if (base < t.every_lo || base + kKvStep > t.every_hi) {
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int tok = mt + 4 * x + e;
            if (tok < mine.lo || tok >= mine.hi) st[x][e] = -kInf;
          }
        // a NaN among the values must reach the rows that see it, and no other:
        // it is taken out of the product, and the rows are found by a product
        // of their view (ones) with the NaNs' places (ones)
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < T; ++i)
          any |= nan_codes(vw[i].x) | nan_codes(vw[i].y) | nan_codes(vw[i].z) | nan_codes(vw[i].w);
        if (__ballot(any != 0)) {
          uint32_t see[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int tok = mt + 2 * k;
            see[k] = (tok >= mine.lo && tok < mine.hi ? 0x3f80u : 0u) |
                     (tok + 1 >= mine.lo && tok + 1 < mine.hi ? 0x3f800000u : 0u);
          }
#pragma unroll
          for (int i = 0; i < T; ++i) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&vw[i]);
            f32x4 hit{0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const uint32_t n0 = nan_codes(w[2 * u]), n1 = nan_codes(w[2 * u + 1]);
              hit = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  frag(ones2<false>(n0), ones2<true>(n0), ones2<false>(n1), ones2<true>(n1)),
                  frag(see[4 * u], see[4 * u + 1], see[4 * u + 2], see[4 * u + 3]), hit, 0, 0, 0);
              w[2 * u] &= ~(n0 | (n0 - (n0 >> 7)));
              w[2 * u + 1] &= ~(n1 | (n1 - (n1 >> 7)));
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (hit[e] > 0.f) o[i][e] = __builtin_nanf("");
          }
        }
      }
      float mx = -kInf;
#pragma unroll
      for (int x = 0; x < 4; ++x) mx = fmaxf(fmaxf(fmaxf(mx, st[x][0]), fmaxf(st[x][1], st[x][2])), st[x][3]);
      mx = max_rows(mx);
      if (__ballot(mx > M + slack)) {
        const float Mn = fmaxf(M, mx);
        const float f = Mn == M ? 1.f : __builtin_amdgcn_exp2f((M - Mn) * cs);
        M = Mn;
        L *= f;
#pragma unroll
        for (int i = 0; i < T; ++i) o[i] *= f;
      }
      const Ref ref(M, cs);
      uint32_t pw[8];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        float p[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) p[e] = ref.p(st[x][e]);
        L += (p[0] + p[1]) + (p[2] + p[3]);
        pw[2 * x] = pack_bf2_hw(p[0], p[1]);
        pw[2 * x + 1] = pack_bf2_hw(p[2], p[3]);
      }
#pragma unroll
      for (int i = 0; i < T; ++i) {
        const bf16x8 lo = frag_fp8(vw[i].x, vw[i].y, vsc), hi = frag_fp8(vw[i].z, vw[i].w, vsc);
        o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(lo, frag(pw[0], pw[1], pw[2], pw[3]), o[i], 0, 0, 0);
        o[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(hi, frag(pw[4], pw[5], pw[6], pw[7]), o[i], 0, 0, 0);
      }
      if (more) load_v();
    }
    L = sum_rows(L);

    // join the waves
    if (g == 0) {
      lds.m[wave][q] = M * cs;
      lds.l[wave][q] = L;
    }
#pragma unroll
    for (int i = 0; i < T; ++i) *reinterpret_cast<f32x4*>(&lds.o[wave][q][16 * i + 4 * g]) = o[i];
    // the next piece's first loads are under way while this one is written
    if (have_next) {
      kid = next_kid, vid = next_vid;
      start(next);
    }
    __syncthreads();
    const int Hq = c.H * a.G;
    for (int i = tid; i < (t.r1 - t.r0 + 1) * (D / 4); i += 64 * kWaves) {
      const int row = i / (D / 4), ch = (i - row * (D / 4)) * 4;
      float top = lds.m[0][row];
#pragma unroll
      for (int w = 1; w < kWaves; ++w) top = fmaxf(top, lds.m[w][row]);
      const float ref = top == -kInf ? 0.f : top;
      float l = 0.f;
      f32x4 v{0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        const float f = __builtin_amdgcn_exp2f(lds.m[w][row] - ref);
        l += lds.l[w][row] * f;
        v += *reinterpret_cast<const f32x4*>(&lds.o[w][row][ch]) * f;
      }
      if (slot >= 0) {
        float* dst = sched_slot(a.work, slot, 16, D);
        *reinterpret_cast<f32x4*>(dst + row * D + ch) = v;
        if (ch == 0) dst[16 * D + row] = top, dst[16 * D + 16 + row] = l;
      } else {
        write_row<D>(a, s, Hq, h, t.r0 + row, ch, v, l, row_sees(c, a, s, t.r0 + row));
      }
    }
    __syncthreads();
    p = next;
    have = have_next;
  }
  pieces.finish();
}

// ----------------------------------------------------------------------------
// Many rows: 128 rows of one (sequence, key/value head), 32 a wave.
// A step's 64 tokens are converted to bf16 once for the workgroup, on the way
// from registers into LDS (two buffers, one barrier a step: the next step's
// codes are converted and the one after's loads issued before the products),
// and every wave runs S^T = K Q^T and O^T = V^T P^T over them with 32x32x16
// products.  As in the few-row kernel the keys' rows are dealt to the matrix
// rows so that a lane's 16 scores of a 32-token tile are 16 tokens in order,
// which are its probabilities in the second product.
//
// A chunk of 2048 tokens over 16301 cached ones (32 query heads on 8, 128
// channels, 581 GFLOP) takes 605 .. 620 us, 940 .. 960 TFLOP/s, where a library
// product of 8192^3 reaches 1200.  Under the counters the clock is down to 1.9
// GHz and the matrix pipes are busy for 45 % of its cycles: what makes the loop
// denser gives little time.
// 64 rows a wave halve the reads from LDS, but take all registers of a SIMD
// for one wave: 894 us when 32 rows took 736.
// ----------------------------------------------------------------------------
typedef float f32x16 __attribute__((ext_vector_type(16)));

__device__ __forceinline__ float max_halves(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(a[0]), __uint_as_float(a[1]));
}
__device__ __forceinline__ float sum_halves(float x) {
  auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
constexpr int kAhead = 8;  // reads of an operand from LDS ahead of its product

template <int D>
struct ManyTile {
  static constexpr int R = 128;
  static constexpr int U = D / 8;                 // 16-byte units of a token's keys in LDS
  static constexpr int G = U % 16 == 0 ? 16 : U % 8 == 0 ? 8 : U % 4 == 0 ? 4 : 2;
  static constexpr int SH = G == 16 ? 0 : G == 8 ? 1 : G == 4 ? 2 : 3;
  static constexpr int T = (D + 31) / 32, DV = 32 * T;
  static constexpr int NP = (D + 63) / 64;        // 16-byte pieces of a lane: a wave brings in one 16-token block
  // workgroups of a CU: what registers (two waves a SIMD) and LDS allow
  static constexpr int PER_CU = D <= 128 ? 2 : 1;
  // Units of a row change places with its number, so that 16 lanes of a
  // read (16 rows, one unit) fall on different banks.
  static __device__ __forceinline__ int k_unit(int row, int u) { return row * U + (u ^ ((row >> SH) & (G - 1))); }
};

template <int D>
struct TileLds {
  typedef ManyTile<D> X;
  uint4 k[2][64 * X::U];
  uint4 v[2][8 * X::DV];        // [16-token block][half][channel]: 8 tokens a unit
  uint32_t mark[2][4 * X::DV];  // [block][channel]: a bit for each token whose value is NaN
  uint32_t bad[2];              // a byte for each block without a page
  // Step with marks, plus 1.  It has no first value, as storing one would race
  // with another wave's first mark; whatever it holds is right, because a step
  // that rows differ in writes all its marks, and unmarked values change nothing.
  int nan[2];
  SchedLds sched;
};

template <int D, bool WHOLE>
__device__ __forceinline__ void tile_part(const KvView& c, const KvAttn& a, const KvSched& d, TileLds<D>& lds) {
  typedef ManyTile<D> X;
  constexpr int T = X::T, NP = X::NP, QF = D / 16;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int q = lane & 31, hf = lane >> 5, B = 1 << c.lb;
  const bool vec = ((reinterpret_cast<uintptr_t>(a.q) | (uintptr_t)(a.rs * 2) | (uintptr_t)(a.hs * 2)) & 15u) == 0;
  const float cs = a.scale * 1.4426950408889634f, slack = fminf(kSlack / cs, kMax);

  // Piece i of this lane: bytes 16 (lane + 64 i) of the block's keys and of its
  // values (both 16 D bytes); its places in LDS.
  int koff[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const int at = lane + 64 * i, x = at / (D / 16), u = at % (D / 16);  // token of the block, unit pair
    koff[i] = X::k_unit(32 * (wave >> 1) + 8 * (x >> 2) + 4 * (wave & 1) + (x & 3), 2 * u);
  }

  typedef Piece<X::R> P;
  bf16x8 qf[QF];
  auto load_q = [&](const P& p) {
    const int r = min(p.t.r0 + wave * 32 + q, p.t.r1), j = r / a.G;
    const uint16_t* src = a.q + (size_t)(p.s.row0 + j) * a.rs + (size_t)(p.h * a.G + r % a.G) * a.hs + 8 * hf;
#pragma unroll
    for (int i = 0; i < QF; ++i) {
      uint4 x{};
      if (vec) {
        x = *reinterpret_cast<const uint4*>(src + 16 * i);
      } else {
        auto two = [&](int e) { return src[16 * i + e] | (uint32_t)src[16 * i + e + 1] << 16; };
        x = uint4{two(0), two(2), two(4), two(6)};
      }
      qf[i] = __builtin_bit_cast(bf16x8, x);
    }
  };
  // Page and scales of this wave's block, one for all its lanes, come by
  // vector loads all the same: a scalar load in flight would have every read
  // from LDS wait for it (they share a counter, and it returns in no order).
  int id_next = 0;
  auto ids = [&](const P& p, int step, int& id) {
    id = c.table[(size_t)p.seq * c.table_stride + min((step * kKvStep + 16 * wave) >> c.lb, c.width - 1)];
  };
  uint4 kr[NP], vr[NP];
  float ks, vs;
  bool bad, vin;
  auto load = [&](const P& p, int step) {
    const int tok = step * kKvStep + 16 * wave;
    const int id = __builtin_amdgcn_readfirstlane(id_next);
    const bool there = (tok >> c.lb) < c.width && (unsigned)id < (unsigned)c.n_blocks, seen = tok < p.t.hi;
    bad = seen && !there;
    vin = seen && there && tok + 16 > p.t.lo;
    const size_t ph = (size_t)(seen && there ? id : 0) * c.H + p.h;
    const size_t at = ((ph << c.lb) + (tok & (B - 1))) * D;
    const uint4 *kp = reinterpret_cast<const uint4*>(c.k + at), *vp = reinterpret_cast<const uint4*>(c.v + at);
    ks = c.k_scale[ph];
    vs = c.v_scale[ph];
#pragma unroll
    for (int i = 0; i < NP; ++i)
      if (64 * i + 63 < D || lane + 64 * i < D) kr[i] = kp[lane + 64 * i], vr[i] = vp[lane + 64 * i];
  };
  Pieces<X::R, WHOLE> pieces(c, a, d, lds.sched);
  P p, next;
  bool have = pieces.next(p);
  if (have) {
    ids(p, p.t.step0 + p.s0, id_next);
    load(p, p.t.step0 + p.s0);
    load_q(p);
  }
  while (have) {
    const Tile<X::R>& t = p.t;
    const KvSeq& s = p.s;
    const int h = p.h, slot = p.slot;
    const bool have_next = pieces.next(next);
    int next_id = 0;
    if (have_next) ids(next, next.t.step0 + next.s0, next_id);
    const int w0 = t.r0 + wave * 32;  // the wave's rows
    const bool active = w0 <= t.r1;
    const Span mine = row_span(c, a, s, min(w0 + q, t.r1) / a.G);
    // what all and what some of the wave's rows see
    const Span wa = row_span(c, a, s, min(w0, t.r1) / a.G), wb = row_span(c, a, s, min(w0 + 31, t.r1) / a.G);

    f32x16 o[T];
    float M = -kInf, L = 0.f;
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) o[i][e] = 0.f;

    auto split = [&](int step) {  // rows differ in what they see of it
      return step * kKvStep < t.every_lo || (step + 1) * kKvStep > t.every_hi;
    };
    auto mark = [&](int step, int buf) {
      if (split(step)) {
        // A NaN among the values must reach the rows that see it, and no
        // other: it is taken out here, and its place marked for the rows.
        uint32_t any = 0;
#pragma unroll
        for (int i = 0; i < NP; ++i)
          if (64 * i + 63 < D || lane + 64 * i < D) {
            uint32_t* w = reinterpret_cast<uint32_t*>(&vr[i]);
            uint32_t at = 0;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t n = nan_codes(w[k]);
              w[k] &= ~(n | (n - (n >> 7)));
              at |= ((n >> 7 & 1) | (n >> 14 & 2) | (n >> 21 & 4) | (n >> 28 & 8)) << (4 * k);
            }
            lds.mark[buf][wave * X::DV + lane + 64 * i] = at;
            any |= at;
          }
        if (any) lds.nan[buf] = step + 1;
      }
      if (lane == 0) reinterpret_cast<uint8_t*>(&lds.bad[buf])[wave] = bad;
    };
    // half a piece from its codes into LDS: j / 4 is the piece, j % 4 which of
    // the keys' and the values' halves
    auto store = [&](int j, int buf) {
      const int i = j / 4, half = j & 1;
      if (64 * i + 63 < D || lane + 64 * i < D) {
        const uint4 w = j & 2 ? vr[i] : kr[i];
        const uint32_t x = half ? w.z : w.x, y = half ? w.w : w.y;
        const float f = j & 2 ? (vin ? vs : 1.f) : ks;
        const uint4 z{kv_bf2<false>(x, f), kv_bf2<true>(x, f), kv_bf2<false>(y, f), kv_bf2<true>(y, f)};
        if (j & 2)
          lds.v[buf][(2 * wave + half) * X::DV + lane + 64 * i] = z;
        else
          lds.k[buf][koff[i] ^ half] = z;
      }
    };
    auto store_all = [&](int buf) {
#pragma unroll
      for (int j = 0; j < 4 * NP; ++j) store(j, buf);
    };

    // a step's loads are issued one step before it goes into LDS, its page id
    // one before that
    const int begin = t.step0 + p.s0, end = t.step0 + p.s1;
    ids(p, begin + 1, id_next);
    mark(begin, 0);
    store_all(0);
    if (begin + 1 < end) load(p, begin + 1);
    ids(p, begin + 2, id_next);
    __syncthreads();
    for (int step = begin; step < end; ++step) {
      const int buf = (step - begin) & 1, base = step * kKvStep;
      const bool run = active && base < wb.hi && base + kKvStep > wa.lo;
      f32x16 st[2];
      // The next step's codes go into the other buffer beside the products
      // (after the last step the old ones do, which nobody reads).
      if (step + 1 < end) mark(step + 1, buf ^ 1);
      if (run) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 16; ++e) st[x][e] = 0.f;
        // Two chains of products.  Reads from LDS run kAhead products ahead of
        // their use and the order is fixed (left alone, the compiler puts each
        // read right before its product, which then waits for it).
        {
          uint4 kf[kAhead];
          auto read = [&](int g) { kf[g % kAhead] = lds.k[buf][X::k_unit(32 * (g & 1) + q, 2 * (g >> 1) + hf)]; };
#pragma unroll
          for (int g = 0; g < kAhead && g < 2 * QF; ++g) read(g);
#pragma unroll
          for (int g = 0; g < 2 * QF; ++g) {
            __builtin_amdgcn_sched_barrier(0);
            st[g & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, kf[g % kAhead]), qf[g >> 1],
                                                                st[g & 1], 0, 0, 0);
            if (g + kAhead < 2 * QF) read(g + kAhead);
#pragma unroll
            for (int j = 4 * NP * g / (2 * QF); j < 4 * NP * (g + 1) / (2 * QF); ++j) store(j, buf ^ 1);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      } else {
        store_all(buf ^ 1);
      }
      if (step + 2 < end) load(p, step + 2);
      ids(p, step + 3, id_next);
      if (run) {
        const uint32_t bads = __builtin_amdgcn_readfirstlane(lds.bad[buf]);
        const int lo = mine.lo - base - 16 * hf, hi = mine.hi - base - 16 * hf;
        if (bads != 0 || base < wb.lo || base + kKvStep > wa.hi) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            const bool none = (bads >> (8 * (2 * x + hf))) & 1;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              if (none) st[x][e] = __builtin_nanf("");
              if (32 * x + e < lo || 32 * x + e >= hi) st[x][e] = -kInf;
            }
          }
        }
        if (split(step) && lds.nan[buf] == step + 1) {
          // the rows that see a marked value: a product of their view (ones)
          // with the marks (ones)
#pragma unroll
          for (int i = 0; i < T; ++i) {
            f32x16 hit;
#pragma unroll
            for (int e = 0; e < 16; ++e) hit[e] = 0.f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const int ch = 32 * i + q;
              const uint32_t mark = ch < D ? lds.mark[buf][(2 * x + hf) * X::DV + ch] : 0;
#pragma unroll
              for (int u = 0; u < 2; ++u) {
                uint32_t see[4], at[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const int b = 8 * u + 2 * k, e = 32 * x + b;
                  see[k] = (e >= lo && e < hi ? 0x3f80u : 0u) | (e + 1 >= lo && e + 1 < hi ? 0x3f800000u : 0u);
                  at[k] = (mark >> b & 1 ? 0x3f80u : 0u) | (mark >> (b + 1) & 1 ? 0x3f800000u : 0u);
                }
                hit = __builtin_amdgcn_mfma_f32_32x32x16_bf16(frag(at[0], at[1], at[2], at[3]),
                                                              frag(see[0], see[1], see[2], see[3]), hit, 0, 0, 0);
              }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e)
              if (hit[e] > 0.f) o[i][e] = __builtin_nanf("");
          }
        }
        float mx = fmaxf(st[0][0], st[1][0]);
#pragma unroll
        for (int e = 1; e < 16; ++e) mx = fmaxf(fmaxf(mx, st[0][e]), st[1][e]);
        mx = max_halves(mx);
        if (__ballot(mx > M + slack)) {
          const float Mn = fmaxf(M, mx);
          const float f = Mn == M ? 1.f : __builtin_amdgcn_exp2f((M - Mn) * cs);
          M = Mn;
          L *= f;
#pragma unroll
          for (int i = 0; i < T; ++i) o[i] *= f;
        }
        // Group c of 8 tokens: its probabilities, then its products, beside which
        // the next group's probabilities are made, and the reads as above.
        {
          const Ref ref(M, cs);
          uint32_t pw[2][4];  // groups c and c + 1
          auto prob = [&](int c, int e) {  // tokens 2 e and 2 e + 1 of group c
            const float p0 = ref.p(st[c >> 1][8 * (c & 1) + 2 * e]), p1 = ref.p(st[c >> 1][8 * (c & 1) + 2 * e + 1]);
            L += p0 + p1;
            pw[c & 1][e] = pack_bf2_hw(p0, p1);
          };
          uint4 vf[kAhead];
          auto read = [&](int g) {
            const int c = g / T, i = g % T;
            vf[g % kAhead] = lds.v[buf][(2 * (2 * (c >> 1) + hf) + (c & 1)) * X::DV + 32 * i + q];
          };
#pragma unroll
          for (int g = 0; g < kAhead && g < 4 * T; ++g) read(g);
#pragma unroll
          for (int e = 0; e < 4; ++e) prob(0, e);
#pragma unroll
          for (int c = 0; c < 4; ++c)
#pragma unroll
            for (int i = 0; i < T; ++i) {
              const int g = c * T + i;
              __builtin_amdgcn_sched_barrier(0);
              o[i] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                  __builtin_bit_cast(bf16x8, vf[g % kAhead]),
                  frag(pw[c & 1][0], pw[c & 1][1], pw[c & 1][2], pw[c & 1][3]), o[i], 0, 0, 0);
              if (g + kAhead < 4 * T) read(g + kAhead);
              if (c < 3)
#pragma unroll
                for (int e = 4 * i / T; e < 4 * (i + 1) / T; ++e) prob(c + 1, e);
            }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      __syncthreads();
    }

    // the next piece's first loads are under way while this one is written
    if (have_next) {
      id_next = next_id;
      load(next, next.t.step0 + next.s0);
      load_q(next);
    }
    const int Hq = c.H * a.G;
    const float l = sum_halves(L);
    const int row = wave * 32 + q, rr = t.r0 + row;
    const bool there = rr <= t.r1;  // (the same in both lanes of a row)
    if (there && slot >= 0) {
      float* dst = sched_slot(a.work, slot, X::R, D);
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int e = 0; e < 16; e += 4) {
          const int ch = 32 * i + 2 * e + 4 * hf;
          if (ch < D)
            *reinterpret_cast<f32x4*>(dst + row * D + ch) = f32x4{o[i][e], o[i][e + 1], o[i][e + 2], o[i][e + 3]};
        }
      if (hf == 0) dst[X::R * D + row] = M * cs, dst[X::R * D + X::R + row] = l;
    } else if (there) {
      // The two halves of the wave hold four channels in turn; they change
      // places so that a lane has eight in a row: half as many stores.
      const float inv = mine.hi > mine.lo ? 1.f / l : 0.f;
      uint16_t* dst = a.out + ((size_t)(s.row0 + rr / a.G) * Hq + h * a.G + rr % a.G) * D + 8 * hf;
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int e = 0; e < 16; e += 8)
          if (32 * i + 2 * e < D) {
            uint32_t x[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const auto z = __builtin_amdgcn_permlane32_swap(
                  pack_bf2_hw(o[i][e + 2 * k] * inv, o[i][e + 2 * k + 1] * inv),
                  pack_bf2_hw(o[i][e + 4 + 2 * k] * inv, o[i][e + 5 + 2 * k] * inv), false, false);
              x[k] = z[0];
              x[2 + k] = z[1];
            }
            *reinterpret_cast<uint4*>(dst + 32 * i + 2 * e) = uint4{x[0], x[1], x[2], x[3]};
          }
    }
    p = next;
    have = have_next;
  }
  pieces.finish();
}

template <int D, bool WHOLE>
__global__ __launch_bounds__(64 * kWaves, WHOLE ? RowsTile<D>::WHOLE_PER_CU : RowsTile<D>::PER_CU) void kv_rows_kernel(
    KvView c, KvAttn a, KvSched d) {
  __shared__ RowsLds<D> lds;
  rows_part<D, WHOLE>(c, a, d, lds);
}

template <int D, bool WHOLE>
__global__ __launch_bounds__(256, ManyTile<D>::PER_CU) void kv_tile_kernel(KvView c, KvAttn a, KvSched d) {
  __shared__ TileLds<D> lds;
  tile_part<D, WHOLE>(c, a, d, lds);
}

template <int R, int D>
__global__ __launch_bounds__(256) void kv_join_kernel(KvView c, KvAttn a, int workers) {
  join_part<R, D>(c, a, workers, blockIdx.x);
}
template <int R, int D>
__global__ __launch_bounds__(256) void kv_join_both_kernel(KvView c, KvAttn a, int workers, KvAttn few_a,
                                                           int few_workers) {
  if ((int)blockIdx.x < workers)
    join_part<R, D>(c, a, workers, blockIdx.x);
  else
    join_part<16, D>(c, few_a, few_workers, blockIdx.x - workers);
}

constexpr int rows_workers(int D) { return D > 128 ? 256 : 512; }
constexpr int tile_workers(int D) { return D > 128 ? 256 : 512; }
// A chunk of 2048 tokens: workgroups 0 .. 255 end at 627 us and the others at
// 768 us with equal parts; at 24 / 256 both ends meet (643 -> 633 us).
constexpr int kSkew = 24;
// 32 sequences of 20 rows: 51 us in the many-row form, 53 us as two 16-row tiles.
constexpr int kFewRows = 16;
// Up to this many steps an item goes to a workgroup whole: no parts to find, no
// pieces to join, and the hardware deals the items.  4 short requests 17.5 us in
// parts, 8.2 us whole; 8 prompts of 240 .. 890 tokens 64 and 49 us; 18 steps (a
// window of 1024, 96 sequences) 22 and 12 us.  Over 120 batches of all kinds the
// time over the floor is 3.6 times with parts alone and 2.26 .. 2.29 at 12, 20
// and 32 steps: past 20 single batches gain or lose up to half.
constexpr int kWholeSteps = 20;

// Steps of an item at most, as far as the host can tell.
int max_steps(const KvView& c, const KvAttn& a) {
  const int64_t cap = ((int64_t)c.width << c.lb) / kKvStep + 1;
  return (int)(a.causal && a.window > 0 ? std::min<int64_t>(cap, ((int64_t)a.window + c.max_new) / kKvStep + 2) : cap);
}

size_t tile_bytes(int D) { return (sched_bytes(tile_workers(D), 128, D) + 255) / 256 * 256; }

// Sequences of at most kFewRows rows (new tokens times query heads of a
// key/value head) take the few-row form, the others the many-row one; each
// is launched unless the batch cannot hold a sequence for it.
template <int D>
hipError_t launch_dim(const KvView& c, const KvAttn& a, hipStream_t stream) {
  constexpr int R = ManyTile<D>::R;
  constexpr int rw = rows_workers(D), tw = tile_workers(D);
  static_assert(rw == 256 * RowsTile<D>::PER_CU && tw == 256 * ManyTile<D>::PER_CU);
  const int64_t rows = (int64_t)c.max_new * a.G, heads = (int64_t)c.n_seq * c.H;
  const bool many = rows > kFewRows;
  // Whether sequences of few rows are left to the few-row form.  In a batch of
  // few sequences with more rows than that on average (prompts, drafts) the
  // many-row form takes them along, which saves a launch that may find nothing:
  // 8 drafts of 3 .. 9 rows 44 -> 27 us, 8 prompts 51 -> 50 us, 2 prompts with 6
  // single rows 84 -> 75 us, a chunk of 1024 with 8 single rows 143 -> 138 us.
  const bool few = !many || (c.n_rows < (int64_t)c.max_new * c.n_seq &&
                             (c.n_seq > 16 || (int64_t)c.n_rows * a.G < kFewRows * (int64_t)c.n_seq));
  const int64_t few_tiles = (std::min<int64_t>(rows, kFewRows) + 15) / 16, tiles = (rows + R - 1) / R;
  KvSched fd{rw == 512 ? 9 : 8, rw == 512 ? kSkew : 0, (int)few_tiles, 2, 6, 0, 8, 0, many ? kFewRows : INT32_MAX};
  KvSched td{tw == 512 ? 9 : 8, tw == 512 ? kSkew : 0, (int)tiles, 3, 6, a.causal, 4, few ? kFewRows : 0, INT32_MAX};

  if (max_steps(c, a) <= kWholeSteps && std::max(few_tiles, many ? tiles : 0) * heads <= 1 << 20) {
    if (few)
      MLORA_LAUNCH("kv_rows", (kv_rows_kernel<D, true>), dim3((unsigned)(few_tiles * heads)), dim3(64 * kWaves), 0,
                   stream, c, a, fd);
    if (many)
      MLORA_LAUNCH("kv_tiles", (kv_tile_kernel<D, true>), dim3((unsigned)(tiles * heads)), dim3(256), 0, stream, c,
                   a, td);
    return launched();
  }
  KvAttn fa = a;
  if (many) fa.work = static_cast<char*>(a.work) + tile_bytes(D);
  if (few) MLORA_LAUNCH("kv_rows", (kv_rows_kernel<D, false>), dim3(rw), dim3(64 * kWaves), 0, stream, c, fa, fd);
  if (many) MLORA_LAUNCH("kv_tiles", (kv_tile_kernel<D, false>), dim3(tw), dim3(256), 0, stream, c, a, td);
  if (few && many)
    MLORA_LAUNCH("kv_join", (kv_join_both_kernel<R, D>), dim3(tw + rw, 8), dim3(256), 0, stream, c, a, tw, fa, rw);
  else if (many)
    MLORA_LAUNCH("kv_join", (kv_join_kernel<R, D>), dim3(tw, 8), dim3(256), 0, stream, c, a, tw);
  else
    MLORA_LAUNCH("kv_join", (kv_join_kernel<16, D>), dim3(rw, 4), dim3(256), 0, stream, c, a, rw);
  return launched();
}

}  // namespace

bool kv_attention_dim(int dim) {
  return dim == 32 || dim == 64 || dim == 80 || dim == 96 || dim == 112 || dim == 128 || dim == 160 || dim == 192 ||
         dim == 256;
}

size_t kv_work_bytes(const KvView& c, int heads) {
  if (c.n_rows == 0) return 0;
  const size_t few = sched_bytes(rows_workers(c.D), 16, c.D);
  return (int64_t)c.max_new * (heads / c.H) > kFewRows ? tile_bytes(c.D) + few : few;
}

hipError_t launch_kv_attention(const KvView& c, const KvAttn& a, hipStream_t stream) {
  switch (c.D) {
    case 32: return launch_dim<32>(c, a, stream);
    case 64: return launch_dim<64>(c, a, stream);
    case 80: return launch_dim<80>(c, a, stream);
    case 96: return launch_dim<96>(c, a, stream);
    case 112: return launch_dim<112>(c, a, stream);
    case 128: return launch_dim<128>(c, a, stream);
    case 160: return launch_dim<160>(c, a, stream);
    case 192: return launch_dim<192>(c, a, stream);
    case 256: return launch_dim<256>(c, a, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace mlora
