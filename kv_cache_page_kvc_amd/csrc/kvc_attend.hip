// kvc_attend.hip -- gfx950 attention over the resident 8-bit cache.
//
// For a query row i and the positions j it sees, with the page scales ks, vs:
//   t_ij = log2(e) * scale * ks[page(j)] * <q_i, kcode_j> + log2(vs[page(j)])
//   w_ij = 2^(t_ij - m_i),  m_i 4 below a running reference of the t_ij
//   out_i = sum_j w_ij vcode_j / sum_j w_ij / vs[page(j)].
// Folding log2(vs) into the exponent makes w the weight of a *code*: V's codes
// then enter the product as they are, and w < 2^16 is a binary16 value
// whatever the pages' scales are.  Both products run on the matrix cores in
// binary16 with binary32 sums: E4M3FN and INT8 codes are binary16 values
// exactly, a query row is scaled by a power of two to a largest |q| in
// [2^14, 2^15), which keeps every BF16 or FP16 value above 2^-29 of that
// exact, and the weights are rounded to 11 significant bits (off by 2^-11 of
// themselves at most, and by 2^-29 of the largest where they are below 2^-18
// of it).  The denominator, the maxima and the merged sums are binary32.
//
// Operands without a transpose.  A wave takes 64 positions at a time as 4
// groups of 16 (a group lies in one page).  Scores are computed transposed, S^T =
// K Q^T, with row 4g + j of product tile i standing for position 16g + 4i + j:
// after 4 tiles lane group g (16 lanes, one query row each) holds the scores
// of the 16 positions of group g, which is exactly the operand layout of the
// second product, out^T = V^T W^T, when V is stored token-minor.  So scores
// and weights stay in registers, a lane's loads are 16 consecutive bytes of K
// (dimensions) and of V (positions), and a row's maximum takes two lane swaps.
//
// attend_kernel, for single tokens, drafts and short calls, is bound by the
// cache's bytes: 64 users of 500 to 8000 positions (557 MB) take 123 us, 4.5
// TB/s, where a copy reaches 5.0.  attend_rows_kernel, for prompts, is bound
// by the vector instructions around the matrix instructions -- an exponential,
// a fused multiply-add, a sum, half a conversion and a maximum a score, of 64
// scores a lane and tile -- and by the waits between them, at 1.1 PFLOP/s on an
// 8192-row prompt (500 us; matrix units 51% busy, vector units 63%), where a
// large binary16 product of the library reaches 1.4.
#include <type_traits>

#include "kvc_cache_device.h"

namespace kvc {
namespace {

constexpr int kTile = 64;             // positions a wave takes at a time
constexpr int kWaves = 4;             // waves of a workgroup of attend_kernel
// A row's reference m is within kSlack below the largest t seen so far, so
// weights are at most 2^(kShift + kSlack), a binary16 value, and sums need a
// new reference only when t has grown by more than kSlack.  Below 2^-14 a
// weight is rounded to a multiple of 2^-24, at most 2^-29 of the largest off:
// 2^-12 for a context of 131,072.  (kShift = 12, kSlack = 3.5 raised the
// reference in a fifth of the half tiles of an 8192-token prompt and cost 4%.)
constexpr float kShift = 4.0f, kSlack = 11.5f;
constexpr _Float16 kMostWeight = 46336.0f;   // 2^15.5
// Page scales below this count as this: an empty page's scale may be 0.  The
// scale rule gives at least 1e-12 / 448.
constexpr float kMinScale = 0x1p-64f;

// 8 codes -> 8 binary16 values, exactly
template <uint32_t CODEC>
__device__ __forceinline__ f16x8 codes_f16(uint32_t lo, uint32_t hi) {
  union { f16x8 v; f16x2 p[4]; } r;
  if constexpr (CODEC == C_FP8) {
    r.p[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.0f, false);
    r.p[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)lo, 1.0f, true);
    r.p[2] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.0f, false);
    r.p[3] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)hi, 1.0f, true);
  } else {
    // byte b + 128 below the exponent of 1024: 1024 + b + 128, less 1152
    const uint32_t w[2] = {lo ^ 0x80808080u, hi ^ 0x80808080u};
    const f16x2 off = {(_Float16)1152.0f, (_Float16)1152.0f};
#pragma unroll
    for (int i = 0; i < 2; i++) {
      r.p[2 * i] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w[i], 0x04010400u)) - off;
      r.p[2 * i + 1] = __builtin_bit_cast(f16x2, __builtin_amdgcn_perm(0x64646464u, w[i], 0x04030402u)) - off;
    }
  }
  return r.v;
}

// bytes [0, n) of 16, the others 0
__device__ __forceinline__ uint4 first_bytes(uint4 v, int n) {
  uint32_t a[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const int k = n - 4 * i;
    a[i] = k >= 4 ? a[i] : (k <= 0 ? 0u : a[i] & ((1u << (8 * k)) - 1u));
  }
  return make_uint4(a[0], a[1], a[2], a[3]);
}

__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Workgroup barrier for LDS only: __syncthreads would also wait for the global
// loads in flight, which are registers of their own wave.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// one row tile of a sequence and KV head
struct Tile {
  Seq s;
  int rows, row0;        // rows of the sequence (token * group + head), first of the tile
  int from, end;         // positions that some row of the tile sees
  int begin;             // `from`, down to a multiple of kTile
  int all_from, all_to;  // positions that every row of the tile sees
};
// the tile of m rows that starts at row0
__device__ __forceinline__ bool make_tile(const AttendParams& p, const Seq& s, int64_t row0, int m, Tile& t) {
  t.s = s;
  if (!t.s.ok) return false;
  const int64_t rows = (int64_t)t.s.n * p.group;
  if (row0 >= rows) return false;
  t.rows = (int)rows;
  t.row0 = (int)row0;
  const int first = t.row0 / (int)p.group, last = min(t.rows - 1, t.row0 + m - 1) / (int)p.group;
  t.end = p.causal ? max(0, min(t.s.len, t.s.start + last + 1)) : t.s.len;
  t.all_to = p.causal ? min(t.s.len, t.s.start + first + 1) : t.s.len;
  t.from = p.window ? max(0, t.s.start + first - (int)p.window + 1) : 0;
  t.begin = t.from / kTile * kTile;
  t.all_from = p.window ? t.s.start + last - (int)p.window + 1 : 0;
  return true;
}

// Query row r (token * group + head) of KV head h as the second operand of
// the score product, this lane's share: the row scaled by a power of two,
// `crow` what its scores then have to be multiplied with (negative: the row
// has a NaN or an infinity, and so no finite softmax), `pos` its position
// (kNowhere: no such row, which sees nothing).
constexpr int kNowhere = -0x40000001;   // below every position; a window less than 2^30 can be taken off it
template <int D>
__device__ __forceinline__ void load_query(const AttendParams& p, const Tile& t, uint32_t h, int r, f16x8* q,
                                           float& crow, int& pos) {
  constexpr int KS = D / 32;
  const int lane = threadIdx.x & 63, g = lane >> 4, G = (int)p.group, i = r / G;
  const bool in = r < t.rows;
  pos = in ? t.s.start + i : kNowhere;
  // a row that is not there loads the first one's values; all loads go out together
  const int row = in ? i : 0, head = in ? r - i * G : 0;
  const uint16_t* qp = p.q.data + (int64_t)(t.s.r0 + row) * p.q.stride_row + (int64_t)((int)h * G + head) * p.q.stride_head;
  uint4 raw[KS];
#pragma unroll
  for (int ks = 0; ks < KS; ks++) raw[ks] = ld_global16(qp + (D >= 64 ? 64 * (ks / 2) + 16 * g + 8 * (ks & 1) : 8 * g));
  float x[KS][8];
  auto unpack = [&](auto dt) {
#pragma unroll
    for (int ks = 0; ks < KS; ks++) {
      const uint32_t a[4] = {raw[ks].x, raw[ks].y, raw[ks].z, raw[ks].w};
#pragma unroll
      for (int j = 0; j < 4; j++) {
        const f32x2 f = unpack2<decltype(dt)::value>(a[j]);
        x[ks][2 * j] = f.x;
        x[ks][2 * j + 1] = f.y;
      }
    }
  };
  if (p.dtype == KVC_BF16) unpack(std::integral_constant<int, KVC_BF16>{});
  else unpack(std::integral_constant<int, KVC_FP16>{});
  float am = 0.0f;
  bool odd = false;
#pragma unroll
  for (int ks = 0; ks < KS; ks++)
#pragma unroll
    for (int j = 0; j < 8; j++) {
      x[ks][j] = in ? x[ks][j] : 0.0f;
      odd |= !(fabsf(x[ks][j]) < __builtin_inff());
      am = fmaxf(am, fabsf(x[ks][j]));
    }
  am = max_across_groups(am);
  const bool bad = max_across_groups(odd ? 1.0f : 0.0f) != 0.0f;
  const int e = am > 0.0f ? 15 - __builtin_amdgcn_frexp_expf(am) : 0;
#pragma unroll
  for (int ks = 0; ks < KS; ks++)
#pragma unroll
    for (int j = 0; j < 8; j++) q[ks][j] = (_Float16)(bad ? 0.0f : ldexpf(x[ks][j], e));
  crow = bad ? -1.0f : ldexpf(p.scale_log2, -e);
}
// Of the positions at .. at + 15, of which `valid` are written, a row at `pos`
// sees at + [lo, hi].
struct Seen {
  int lo, hi;
};
__device__ __forceinline__ Seen seen(const AttendParams& p, int pos, int at, int valid) {
  const int rel = pos - at;
  return {p.window ? rel - (int)p.window + 1 : 0, pos == kNowhere ? -1 : min(valid - 1, p.causal ? rel : 15)};
}

// What a score of this lane's group is multiplied with.  It is kept positive,
// so that the -infinity of a hidden score stays one whatever the scales are.
__device__ __forceinline__ float score_factor(float ks, float crow) {
  return fmaxf(ks * fabsf(crow), 0x1p-126f);
}

// The row's result: o holds dimensions 16 n + 4 g .. + 3, m and l are the row's.
template <int D>
__device__ __forceinline__ void store_row(const AttendParams& p, const Tile& t, uint32_t h, int split, int r,
                                          const f32x4* o, float crow, float m, float l) {
  constexpr int NV = D / 16;
  if (r >= t.rows) return;
  if (crow < 0.0f && l != 0.0f) l = __builtin_nanf("");
  const int g = (threadIdx.x & 63) >> 4, G = (int)p.group, Hq = (int)p.c.heads * G;
  const int row = t.s.r0 + r / G, head = (int)h * G + r % G;
  if (p.splits > 1) {
    const int64_t slots = (int64_t)p.b.n_rows * Hq;      // (row, query head) pairs of a split
    const int64_t at = split * slots + (int64_t)row * Hq + head;
    float* acc = p.ws + at * D;
#pragma unroll
    for (int n = 0; n < NV; n++) *(f32x4*)(acc + 16 * n + 4 * g) = o[n];
    if (g == 0) {
      float* ml = p.ws + p.splits * slots * D + at * 2;
      ml[0] = m;
      ml[1] = l;
    }
    return;
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* dst = p.out.data + (int64_t)row * p.out.stride_row + (int64_t)head * p.out.stride_head;
  auto put = [&](auto dt) {
#pragma unroll
    for (int n = 0; n < NV; n++) {
      const f32x4 y = o[n] * inv;
      st_global8(dst + 16 * n + 4 * g, make_uint2(pack2<decltype(dt)::value>(y[0], y[1]), pack2<decltype(dt)::value>(y[2], y[3])));
    }
  };
  if (p.dtype == KVC_BF16) put(std::integral_constant<int, KVC_BF16>{});
  else put(std::integral_constant<int, KVC_FP16>{});
  if (p.lse && g == 0)
    p.lse[(int64_t)row * Hq + head] =
        l == 0.0f ? -__builtin_inff() : (m - kShift + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
}

// D: head size; NT: tile of 16 * NT query rows, the same for the workgroup's
// four waves, which take the context's tiles in turn and are joined in LDS.
template <int D, int NT, uint32_t CODEC>
__global__ __launch_bounds__(64 * kWaves, 2) void attend_kernel(AttendParams p) {
  constexpr int M = 16 * NT, KS = D / 32, NV = D / 16, CH = D >= 64 ? D / 64 : 1;
  constexpr bool HOIST = D * NT <= 128;     // a tile's V loads go out with its K loads: room for both in registers
  __shared__ float s_acc[kWaves / 2][M][D + 4];
  __shared__ float s_m[kWaves][M], s_l[kWaves][M];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, c = lane & 15;
  const uint32_t H = p.c.heads, h = blockIdx.x % H, rest = blockIdx.x / H;
  const int split = (int)(rest % p.splits);
  Tile t;
  const Seq seq = seq_of_unit(p.b, rest / p.splits);
  if (!make_tile(p, seq, (int64_t)seq.unit * M, M, t)) return;
  const int T = 1 << p.c.tshift;
  // this split's positions; the first one also stands for a tile that sees nothing
  const int64_t from0 = t.begin + (int64_t)split * p.chunk;
  if (split && from0 >= t.end) return;
  const int lo = (int)(from0 / kTile), hi = (int)min((int64_t)t.end, from0 + p.chunk);

  f16x8 q[NT][KS];
  float crow[NT], m[NT], l[NT];
  int pos[NT];
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    load_query<D>(p, t, h, t.row0 + 16 * nt + c, q[nt], crow[nt], pos[nt]);
    m[nt] = -__builtin_inff();
    l[nt] = 0.0f;
  }
  f32x4 o[NT][NV];
#pragma unroll
  for (int nt = 0; nt < NT; nt++)
#pragma unroll
    for (int n = 0; n < NV; n++) o[nt][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  const int32_t* table = p.b.table + (int64_t)t.s.b * p.b.stride_table;
  const int last_group = (t.s.len - 1) >> 4;
  bool bad_page = false;
  const uint8_t* k_lane = p.c.k_codes + (uint64_t)h * T * D + (c & 3) * D + (D >= 64 ? 16 * g : 8 * g);
  const uint8_t* v_lane = p.c.v_codes + (uint64_t)h * T * D + c * T;
  // page ids of a tile: of this lane's group (scores, V) and of the group of its K rows
  auto page_ids = [&](int tile, int32_t& v, int32_t& k) {
    v = table[(16 * min(4 * tile + g, last_group)) >> p.c.tshift];
    k = table[(16 * min(4 * tile + (c >> 2), last_group)) >> p.c.tshift];
  };
  int32_t next_v = 0, next_k = 0;
  if ((lo + wave) * kTile < hi) page_ids(lo + wave, next_v, next_k);
  for (int tile = lo + wave; tile * kTile < hi; tile += kWaves) {
    const int base = tile * kTile;
    int32_t pv = next_v, pk = next_k;
    page_ids(tile + kWaves, next_v, next_k);                // used one tile later
    const bool okv = pv >= 0 && (uint32_t)pv < p.c.num_pages, okk = pk >= 0 && (uint32_t)pk < p.c.num_pages;
    bad_page |= !okv & (base + 16 * g + 15 >= t.from) & (base + 16 * g < t.end);   // where a row looks
    pv = okv ? pv : 0;
    pk = okk ? pk : 0;
    const int gv = (16 * min(4 * tile + g, last_group)) & (T - 1);
    const int gk = (16 * min(4 * tile + (c >> 2), last_group)) & (T - 1);
    const uint8_t* kp = k_lane + ((uint64_t)(uint32_t)pk * p.c.stride_page + (uint32_t)(gk * D));
    const uint8_t* vp = v_lane + ((uint64_t)(uint32_t)pv * p.c.stride_page + (uint32_t)gv);
    uint4 kr[4][CH], vr[NV];
#pragma unroll
    for (int i = 0; i < 4; i++)
#pragma unroll
      for (int ch = 0; ch < CH; ch++) {
        if constexpr (D >= 64) {
          kr[i][ch] = ld_global16(kp + 4 * i * D + 64 * ch);
        } else {
          const uint2 w = ld_global8(kp + 4 * i * D);
          kr[i][ch] = make_uint4(w.x, w.y, 0, 0);
        }
      }
    const uint64_t at = (uint64_t)(uint32_t)pv * p.c.stride_scale + h;
    const float ks = p.c.k_scales[at], vs = fmaxf(p.c.v_scales[at], kMinScale);
    if constexpr (HOIST)
#pragma unroll
      for (int n = 0; n < NV; n++) vr[n] = ld_global16(vp + 16 * n * T);
    const int valid = okv ? min(max(t.s.len - base - 16 * g, 0), 16) : 0;   // positions of the group that are written
    const float lvs = __builtin_amdgcn_logf(vs), ivs = __builtin_amdgcn_rcpf(vs);

    f32x4 sc[NT][4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
#pragma unroll
      for (int nt = 0; nt < NT; nt++) sc[nt][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int ch = 0; ch < CH; ch++) {
        const uint4 w = kr[i][ch];
        const f16x8 a0 = codes_f16<CODEC>(w.x, w.y);
#pragma unroll
        for (int nt = 0; nt < NT; nt++) sc[nt][i] = mfma(a0, q[nt][2 * ch], sc[nt][i]);
        if constexpr (D >= 64) {
          const f16x8 a1 = codes_f16<CODEC>(w.z, w.w);
#pragma unroll
          for (int nt = 0; nt < NT; nt++) sc[nt][i] = mfma(a1, q[nt][2 * ch + 1], sc[nt][i]);
        }
      }
    }

    const bool masked = base < t.all_from || base + kTile > t.all_to || __any(valid < 16);
    f16x8 w[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; nt++) {
      const float kc = score_factor(ks, crow[nt]);
      if (masked) {
        const Seen v = seen(p, pos[nt], base + 16 * g, valid);
#pragma unroll
        for (int e = 0; e < 16; e++)
          sc[nt][e >> 2][e & 3] = ((e >= v.lo) & (e <= v.hi)) ? sc[nt][e >> 2][e & 3] : -__builtin_inff();
      }
      float mx = sc[nt][0][0];
#pragma unroll
      for (int e = 1; e < 16; e++) mx = fmaxf(mx, sc[nt][e >> 2][e & 3]);
      const float now = fmaxf(m[nt], max_across_groups(fmaf(mx, kc, lvs)));
      const float ref = now == -__builtin_inff() ? 0.0f : now - kShift;   // a row that has seen nothing yet
      const float keep = now == -__builtin_inff() ? 1.0f : __builtin_amdgcn_exp2f(m[nt] - now);
      m[nt] = now;
      const float shift = lvs - ref;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; i++)
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const float e = __builtin_amdgcn_exp2f(fmaf(sc[nt][i][j], kc, shift));
          sum += e;
          w[nt][i >> 1][4 * (i & 1) + j] = (_Float16)e;
        }
      l[nt] = fmaf(l[nt], keep, sum * ivs);
#pragma unroll
      for (int n = 0; n < NV; n++) o[nt][n] *= keep;
    }

#pragma unroll
    for (int n = 0; n < NV; n++) {
      uint4 v = HOIST ? vr[n] : ld_global16(vp + 16 * n * T);
      if (masked) v = first_bytes(v, valid);   // codes of unwritten positions may be anything, NaN included
      const f16x8 a0 = codes_f16<CODEC>(v.x, v.y), a1 = codes_f16<CODEC>(v.z, v.w);
#pragma unroll
      for (int nt = 0; nt < NT; nt++) {
        o[nt][n] = mfma(a0, w[nt][0], o[nt][n]);
        o[nt][n] = mfma(a1, w[nt][1], o[nt][n]);
      }
    }
  }
  if (__any(bad_page)) flag_seq(p.b, t.s.b, KVC_SEQ_BAD_PAGE);

  // join the waves: every wave brings its sums to the common maximum, then
  // the upper half of the waves adds into the lower half, twice
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    l[nt] = sum_across_groups(l[nt]);
    if (g == 0) {
      s_m[wave][16 * nt + c] = m[nt];
      s_l[wave][16 * nt + c] = l[nt];
    }
  }
  __syncthreads();
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    float top = -__builtin_inff();
#pragma unroll
    for (int v = 0; v < kWaves; v++) top = fmaxf(top, s_m[v][16 * nt + c]);
    float sum = 0.0f;
#pragma unroll
    for (int v = 0; v < kWaves; v++) {
      // a wave that saw nothing has sum 0 (and maximum -inf); a NaN sum stays one
      const float lv = s_l[v][16 * nt + c];
      sum += lv == 0.0f ? 0.0f : lv * __builtin_amdgcn_exp2f(s_m[v][16 * nt + c] - top);
    }
    const float f = l[nt] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m[nt] - top);
    m[nt] = top;
    l[nt] = sum;
#pragma unroll
    for (int n = 0; n < NV; n++) o[nt][n] *= f;
  }
#pragma unroll
  for (int half = kWaves / 2; half >= 1; half /= 2) {
    if (wave >= half && wave < 2 * half)
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int n = 0; n < NV; n++)
          *(f32x4*)&s_acc[wave - half][16 * nt + c][16 * n + 4 * g] = o[nt][n];
    __syncthreads();
    if (wave < half)
#pragma unroll
      for (int nt = 0; nt < NT; nt++)
#pragma unroll
        for (int n = 0; n < NV; n++)
          o[nt][n] += *(const f32x4*)&s_acc[wave][16 * nt + c][16 * n + 4 * g];
    __syncthreads();
  }
  if (wave != 0) return;
#pragma unroll
  for (int nt = 0; nt < NT; nt++) store_row<D>(p, t, h, split, t.row0 + 16 * nt + c, o[nt], crow[nt], m[nt], l[nt]);
}

// Many rows: every wave of the workgroup has 16 * NT rows of its own, and the
// context's tiles go through LDS, converted to binary16 once for all of them.
// LDS holds operand fragments in the order the lanes read them (64 lanes x 16
// bytes each), so neither side has bank conflicts; while tiles are worked on,
// the codes of a later one are on their way into registers, and they are
// converted into the other half of the ring.  Waves 0 .. 3 stage a tile's K,
// each one product tile of 16 positions, waves 4 .. 7 its V.
// At D = 128 twelve waves, three a SIMD, hide each other's latencies best: an
// 8192-row prompt of 32 heads took 522 us, with eight waves and fragments read
// a phase ahead 529 (chunks of INT8: 519 against 556).  Eight waves of 48 rows,
// which read a third less from LDS, took 600 and 602, products of 32 x 32
// scores with half the matrix instructions 577 and 597: neither LDS nor the
// matrix units are what it waits for.
template <int D, int NT, uint32_t CODEC>
__global__ __launch_bounds__(64 * attend_row_waves(D), attend_row_waves(D) * attend_row_resident(D) / 4)
void attend_rows_kernel(AttendParams p) {
  constexpr int M = 16 * NT * attend_row_waves(D), KS = D / 32, NV = D / 16, CH = D >= 64 ? D / 64 : 1;
  constexpr int V0 = 4 * KS;           // V's fragments come behind K's
  // A ring of tiles: half of them are worked on between two barriers while
  // the other half is filled.  Two tiles a barrier where LDS holds four.
  constexpr int RING = D <= 128 ? 4 : 2, AHEAD = RING / 2;
  __shared__ uint4 s_f[RING][V0 + 2 * NV][64];
  __shared__ float4 s_scale[RING][4];  // of each group: K's scale, log2 and reciprocal of V's, written positions
  const int lane = threadIdx.x & 63, g = lane >> 4, c = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), part = wave & 3;
  const bool of_v = wave >= 4, idle = wave >= 8 || (of_v && part >= NV);
  // the last tiles see most (causal): they go first, but for the host's turn of some
  const uint32_t H = p.c.heads, h = blockIdx.x % H, rest = blockIdx.x / H;
  const int split = (int)(rest % p.splits);
  uint32_t turn = rest / p.splits;
  if (turn - p.turn_at < p.turn_at) {
    turn += p.turn;
    if (turn >= 2 * p.turn_at) turn -= p.turn_at;
  }
  Tile t;
  const Seq seq = seq_of_unit(p.b, p.units - 1 - turn);
  if (!make_tile(p, seq, (int64_t)seq.unit * M, M, t)) return;
  const int T = 1 << p.c.tshift, G = (int)p.group;
  const int64_t from0 = t.begin + (int64_t)split * p.chunk;
  if (split && from0 >= t.end) return;
  const int lo = (int)(from0 / kTile), hi = (int)min((int64_t)t.end, from0 + p.chunk);

  f16x8 q[NT][KS];
  float crow[NT], m[NT], l[NT];
  int pos[NT];
  const int row0 = t.row0 + 16 * NT * wave;
#pragma unroll
  for (int nt = 0; nt < NT; nt++) {
    load_query<D>(p, t, h, row0 + 16 * nt + c, q[nt], crow[nt], pos[nt]);
    m[nt] = -__builtin_inff();
    l[nt] = 0.0f;
  }
  f32x4 o[NT][NV];
#pragma unroll
  for (int nt = 0; nt < NT; nt++)
#pragma unroll
    for (int n = 0; n < NV; n++) o[nt][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // positions that some, and that every, row of the wave sees
  const int first = t.s.start + row0 / G, last = t.s.start + min(t.rows - 1, row0 + 16 * NT - 1) / G;
  const bool any_row = row0 < t.rows;
  const int w_begin = p.window ? first - (int)p.window + 1 : 0, w_from = p.window ? last - (int)p.window + 1 : 0;
  const int w_end = any_row ? (p.causal ? last + 1 : t.s.len) : 0, w_to = p.causal ? first + 1 : t.s.len;

  const int32_t* table = p.b.table + (int64_t)t.s.b * p.b.stride_table;
  const int last_group = (t.s.len - 1) >> 4;
  bool bad_page = false;
  // this lane's group of a tile: of its K rows' positions, or of its V columns' (and of its scores')
  const int my_group = of_v ? g : c >> 2;
  auto page_id = [&](int tile) { return table[(16 * min(4 * tile + my_group, last_group)) >> p.c.tshift]; };
  // this wave's share of a tile's codes, and the scales of this lane's group
  uint4 raw[CH];
  float ks_in = 0.0f, vs_in = 0.0f;
  int valid_in = 16;
  const uint8_t* lane_codes = of_v ? p.c.v_codes + (uint64_t)h * T * D + (uint32_t)((16 * part + c) * T)
                                   : p.c.k_codes + (uint64_t)h * T * D + (4 * part + (c & 3)) * D + (D >= 64 ? 16 : 8) * g;
  const uint32_t token_bytes = of_v ? 1 : D, step = of_v ? 64 * T : 64;
  auto load_codes = [&](int tile, int32_t id) {
    if (idle) return;
    const bool ok = (uint32_t)id < p.c.num_pages;
    const uint32_t page = ok ? (uint32_t)id : 0u;
    const uint32_t at = (uint32_t)(16 * min(4 * tile + my_group, last_group)) & (T - 1);
    const uint8_t* src = lane_codes + ((uint64_t)page * p.c.stride_page + at * token_bytes);
#pragma unroll
    for (int ch = 0; ch < CH; ch++) {
      if (D >= 64 || of_v) {
        raw[ch] = ld_global16(src + ch * step);
      } else {
        const uint2 w = ld_global8(src);
        raw[ch] = make_uint4(w.x, w.y, 0, 0);
      }
    }
    if (of_v) {
      const int at_group = tile * kTile + 16 * g;
      bad_page |= !ok & (at_group + 15 >= t.from) & (at_group < t.end);      // where a row looks
      valid_in = ok ? min(max(t.s.len - tile * kTile - 16 * g, 0), 16) : 0;
      if (part == 0) {
        const uint64_t i = (uint64_t)page * p.c.stride_scale + h;
        ks_in = p.c.k_scales[i];
        vs_in = p.c.v_scales[i];
      }
    }
  };
  auto store_codes = [&](int buf) {
    if (idle) return;
    if (of_v && __any(valid_in < 16))
#pragma unroll
      for (int ch = 0; ch < CH; ch++) raw[ch] = first_bytes(raw[ch], valid_in);
#pragma unroll
    for (int ch = 0; ch < CH; ch++) {
      // fragments of K: chunk by chunk of the positions' dimensions; of V: every fourth 16 dimensions
      const int slot = of_v ? V0 + 2 * (part + 4 * ch) : part * KS + (D >= 64 ? 2 * ch : 0);
      *(f16x8*)&s_f[buf][slot][lane] = codes_f16<CODEC>(raw[ch].x, raw[ch].y);
      if (D >= 64 || of_v) *(f16x8*)&s_f[buf][slot + 1][lane] = codes_f16<CODEC>(raw[ch].z, raw[ch].w);
    }
    // through LDS: as registers carried over the loop, the scales would be
    // waited for as soon as they were asked for
    if (wave == 4 && c == 0) {
      const float vc = fmaxf(vs_in, kMinScale);
      s_scale[buf][g] = make_float4(ks_in, __builtin_amdgcn_logf(vc), __builtin_amdgcn_rcpf(vc), (float)valid_in);
    }
  };

  if (lo * kTile < hi) {
    int32_t next = page_id(lo);
#pragma unroll
    for (int i = 0; i < AHEAD; i++) {
      load_codes(lo + i, next);
      next = page_id(lo + i + 1);
      store_codes(i);
    }
    load_codes(lo + AHEAD, next);
    next = page_id(lo + AHEAD + 1);
    for (int tile = lo, buf = 0; tile * kTile < hi; tile++, buf = (buf + 1) % RING) {
      const int base = tile * kTile;
      // the tiles of this half of the ring are in place, and the other half is free
      if (buf % AHEAD == 0) lds_barrier();
      if (base < w_end && base + kTile > w_begin) {
        const float4 group = s_scale[buf][g];
        const float ks = group.x, lvs = group.y, ivs = group.z;
        const int valid = (int)group.w;
        const bool masked = base < w_from || base + kTile > w_to || __any(valid < 16);
        float kc[NT];
#pragma unroll
        for (int nt = 0; nt < NT; nt++) kc[nt] = score_factor(ks, crow[nt]);
        // A tile whose positions every row sees, once every row has a reference:
        // the weights are formed against it as it is, and only if one of them
        // is too large for binary16 is it raised.  Else the maximum comes first.
        bool first = masked;
#pragma unroll
        for (int nt = 0; nt < NT; nt++) first |= m[nt] == -__builtin_inff();
        first = __any(first);
#pragma unroll 1
        for (int hh = 0; hh < 2; hh++) {
          f32x4 sc[NT][2];
#pragma unroll
          for (int i = 0; i < 2; i++)
#pragma unroll
            for (int s = 0; s < KS; s++) {
              const f16x8 a = *(const f16x8*)&s_f[buf][(2 * hh + i) * KS + s][lane];
#pragma unroll
              for (int nt = 0; nt < NT; nt++)
                sc[nt][i] = mfma(a, q[nt][s], s ? sc[nt][i] : f32x4{0.0f, 0.0f, 0.0f, 0.0f});
            }
          f16x8 w[NT];
          float sum[NT];
          auto weigh = [&]() {
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
              const float shift = lvs - (m[nt] - kShift);
              sum[nt] = 0.0f;
#pragma unroll
              for (int e = 0; e < 8; e++) {
                const float y = __builtin_amdgcn_exp2f(fmaf(sc[nt][e >> 2][e & 3], kc[nt], shift));
                sum[nt] += y;
                w[nt][e] = (_Float16)y;
              }
            }
          };
          bool raise = first;
          if (!first) {
            weigh();
            f16x2 top = {0, 0};
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
              const f16x8 x = w[nt];
              const f16x2 a = {x[0], x[1]}, b = {x[2], x[3]}, c2 = {x[4], x[5]}, d = {x[6], x[7]};
              top = __builtin_elementwise_max(top, __builtin_elementwise_max(__builtin_elementwise_max(a, b),
                                                                             __builtin_elementwise_max(c2, d)));
            }
            raise = __any((top[0] > kMostWeight) | (top[1] > kMostWeight));
          }
          if (raise) {
            if (masked)
#pragma unroll
              for (int nt = 0; nt < NT; nt++) {
                const Seen v = seen(p, pos[nt], base + 16 * g + 8 * hh, valid - 8 * hh);
#pragma unroll
                for (int e = 0; e < 8; e++)
                  sc[nt][e >> 2][e & 3] = ((e >= v.lo) & (e <= v.hi)) ? sc[nt][e >> 2][e & 3] : -__builtin_inff();
              }
#pragma unroll
            for (int nt = 0; nt < NT; nt++) {
              float x = sc[nt][0][0];
#pragma unroll
              for (int e = 1; e < 8; e++) x = fmaxf(x, sc[nt][e >> 2][e & 3]);
              const float mx = max_across_groups(fmaf(x, kc[nt], lvs)), now = mx > m[nt] + kSlack ? mx : m[nt];
              const float keep = now == m[nt] ? 1.0f : __builtin_amdgcn_exp2f(m[nt] - now);
              m[nt] = now;
              l[nt] *= keep;
#pragma unroll
              for (int n = 0; n < NV; n++) o[nt][n] *= keep;
            }
            weigh();
            // a row that has seen nothing yet: 2^(-inf + inf)
#pragma unroll
            for (int nt = 0; nt < NT; nt++)
              if (m[nt] == -__builtin_inff()) {
                sum[nt] = 0.0f;
#pragma unroll
                for (int e = 0; e < 8; e++) w[nt][e] = (_Float16)0.0f;
              }
          }
#pragma unroll
          for (int nt = 0; nt < NT; nt++) l[nt] = fmaf(sum[nt], ivs, l[nt]);
#pragma unroll
          for (int n = 0; n < NV; n++) {
            const f16x8 a = *(const f16x8*)&s_f[buf][V0 + 2 * n + hh][lane];
#pragma unroll
            for (int nt = 0; nt < NT; nt++) o[nt][n] = mfma(a, w[nt], o[nt][n]);
          }
        }
      }
      if (base + AHEAD * kTile < hi) {
        store_codes((buf + AHEAD) % RING);
        load_codes(tile + AHEAD + 1, next);
        next = page_id(tile + AHEAD + 2);
      }
    }
  }
  if (__any(bad_page)) flag_seq(p.b, t.s.b, KVC_SEQ_BAD_PAGE);
#pragma unroll
  for (int nt = 0; nt < NT; nt++)
    store_row<D>(p, t, h, split, row0 + 16 * nt + c, o[nt], crow[nt], m[nt], sum_across_groups(l[nt]));
}

// Joins the context splits of one row and query head, one workgroup of WAVES
// each: the lanes take the splits' maxima and sums, then each wave adds up its
// share of the splits' partial sums, eight loads in flight (3 rows x 4 heads of
// 256 splits: 7.5 us with sixteen waves; four took 11.5 for 512).
template <int D, int M, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void attend_join_kernel(AttendParams p, BatchView rows) {
  constexpr int E = D >= 64 ? D / 64 : 1;                 // dimensions of a lane
  __shared__ float s_y[WAVES][D], s_f[kMaxSplits];
  __shared__ float s_top[WAVES], s_sum[WAVES];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int G = (int)p.group, Hq = (int)p.c.heads * G;
  const int head = (int)(blockIdx.x % Hq);
  const Seq seq = seq_of_unit(rows, blockIdx.x / Hq);
  Tile t;
  const int64_t r = (int64_t)seq.unit * G + head % G;
  if (!make_tile(p, seq, r / M * M, M, t) || r >= t.rows) return;
  const int n = t.end > t.begin ? min((int)((t.end - t.begin + (int64_t)p.chunk - 1) / p.chunk), (int)p.splits) : 1;
  const int64_t slots = (int64_t)p.b.n_rows * Hq;
  const int64_t at0 = (int64_t)(seq.r0 + (int)seq.unit) * Hq + head;
  const float* ml = p.ws + p.splits * slots * D + at0 * 2;
  float top = -__builtin_inff();
  for (int s = threadIdx.x; s < n; s += 64 * WAVES) top = fmaxf(top, ml[s * slots * 2]);
  top = wave_fmax(top);
  if (lane == 0) s_top[wave] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WAVES; w++) top = fmaxf(top, s_top[w]);
  float sum = 0.0f;
  for (int s = threadIdx.x; s < n; s += 64 * WAVES) {
    const float m = ml[s * slots * 2], l = ml[s * slots * 2 + 1];
    const float f = l == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m - top);   // a split that saw nothing has sum 0
    s_f[s] = f;
    sum += l == 0.0f ? 0.0f : l * f;
  }
  sum = wave_fsum(sum);
  if (lane == 0) s_sum[wave] = sum;
  __syncthreads();
  float l = 0.0f;
#pragma unroll
  for (int w = 0; w < WAVES; w++) l += s_sum[w];
  float y[E] = {};
  const float* acc = p.ws + at0 * D + (lane < D / E ? lane * E : 0);
#pragma unroll 8
  for (int s = wave; s < n; s += WAVES) {
    const float f = s_f[s];
#pragma unroll
    for (int e = 0; e < E; e++) y[e] = fmaf(acc[s * slots * D + e], f, y[e]);
  }
  if (lane < D / E)
#pragma unroll
    for (int e = 0; e < E; e++) s_y[wave][lane * E + e] = y[e];
  __syncthreads();
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  uint16_t* dst = p.out.data + (int64_t)(seq.r0 + (int)seq.unit) * p.out.stride_row + (int64_t)head * p.out.stride_head;
  for (int d = threadIdx.x; d < D; d += 64 * WAVES) {
    float v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; w++) v += s_y[w][d];
    dst[d] = (uint16_t)(p.dtype == KVC_BF16 ? pack2<KVC_BF16>(v * inv, 0.0f) : pack2<KVC_FP16>(v * inv, 0.0f));
  }
  if (p.lse && threadIdx.x == 0)
    p.lse[at0] = l == 0.0f ? -__builtin_inff() : (top - kShift + __builtin_amdgcn_logf(l)) * 0.693147180559945309f;
}

// The same for few splits, one wave a row and query head: everything it needs
// is asked for at once, and every lane forms the row's maximum and sum.
constexpr uint32_t kFewSplits = 16;
template <int D, int M>
__global__ __launch_bounds__(256) void attend_join_few_kernel(AttendParams p, BatchView rows) {
  constexpr int E = D >= 64 ? D / 64 : 1;                 // dimensions of a lane
  const int lane = threadIdx.x & 63;
  const int G = (int)p.group, Hq = (int)p.c.heads * G;
  const uint32_t id = blockIdx.x * 4 + (uint32_t)__builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  if (id >= p.join_units * (uint32_t)Hq) return;
  const int head = (int)(id % Hq);
  const Seq seq = seq_of_unit(rows, id / Hq);
  Tile t;
  const int64_t r = (int64_t)seq.unit * G + head % G;
  if (!make_tile(p, seq, r / M * M, M, t) || r >= t.rows) return;
  const int n = t.end > t.begin ? min((int)((t.end - t.begin + (int64_t)p.chunk - 1) / p.chunk), (int)p.splits) : 1;
  const int64_t slots = (int64_t)p.b.n_rows * Hq, at0 = (int64_t)(seq.r0 + (int)seq.unit) * Hq + head;
  const float* ml = p.ws + p.splits * slots * D + at0 * 2;
  const float* acc = p.ws + at0 * D + (lane < D / E ? lane * E : 0);
  float m[kFewSplits], l[kFewSplits], y[kFewSplits][E];
#pragma unroll
  for (int s = 0; s < (int)kFewSplits; s++)
    if (s < n) {
      m[s] = ml[s * slots * 2];
      l[s] = ml[s * slots * 2 + 1];
#pragma unroll
      for (int e = 0; e < E; e++) y[s][e] = acc[s * slots * D + e];
    }
  float top = -__builtin_inff(), sum = 0.0f, v[E] = {};
#pragma unroll
  for (int s = 0; s < (int)kFewSplits; s++)
    if (s < n) top = fmaxf(top, m[s]);
#pragma unroll
  for (int s = 0; s < (int)kFewSplits; s++)
    if (s < n) {
      const float f = l[s] == 0.0f ? 0.0f : __builtin_amdgcn_exp2f(m[s] - top);   // a split that saw nothing has sum 0
      sum += l[s] == 0.0f ? 0.0f : l[s] * f;
#pragma unroll
      for (int e = 0; e < E; e++) v[e] = fmaf(y[s][e], f, v[e]);
    }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  uint16_t* dst = p.out.data + (int64_t)(seq.r0 + (int)seq.unit) * p.out.stride_row + (int64_t)head * p.out.stride_head;
  if (lane < D / E)
#pragma unroll
    for (int e = 0; e < E; e++)
      dst[lane * E + e] = (uint16_t)(p.dtype == KVC_BF16 ? pack2<KVC_BF16>(v[e] * inv, 0.0f) : pack2<KVC_FP16>(v[e] * inv, 0.0f));
  if (p.lse && lane == 0)
    p.lse[at0] = sum == 0.0f ? -__builtin_inff() : (top - kShift + __builtin_amdgcn_logf(sum)) * 0.693147180559945309f;
}

template <int D, int NT, bool ROWS>
hipError_t launch_codec(const AttendParams& p, uint32_t codec, hipStream_t stream) {
  constexpr int M = 16 * NT * (ROWS ? attend_row_waves(D) : 1);
  const dim3 grid(p.units * p.splits * p.c.heads);
  if constexpr (ROWS) {
    if (codec == C_FP8) attend_rows_kernel<D, NT, C_FP8><<<grid, 64 * attend_row_waves(D), 0, stream>>>(p);
    else attend_rows_kernel<D, NT, C_INT8><<<grid, 64 * attend_row_waves(D), 0, stream>>>(p);
  } else {
    if (codec == C_FP8) attend_kernel<D, NT, C_FP8><<<grid, 64 * kWaves, 0, stream>>>(p);
    else attend_kernel<D, NT, C_INT8><<<grid, 64 * kWaves, 0, stream>>>(p);
  }
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && p.splits > 1) {
    const uint32_t rows = p.join_units * p.c.heads * p.group;
    if (p.splits <= kFewSplits) attend_join_few_kernel<D, M><<<(rows + 3) / 4, 256, 0, stream>>>(p, p.join);
    else attend_join_kernel<D, M, 16><<<rows, 1024, 0, stream>>>(p, p.join);
    e = hipGetLastError();
  }
  return e;
}
template <int D>
hipError_t launch_tile(const AttendParams& p, uint32_t codec, uint32_t rows, hipStream_t stream) {
  constexpr int M = attend_tile_rows(D);
  if (rows == 16) return launch_codec<D, 1, false>(p, codec, stream);
  if constexpr (D < 256)
    if (rows == 32) return launch_codec<D, 2, false>(p, codec, stream);
  if (rows == M) return launch_codec<D, M / (16 * attend_row_waves(D)), true>(p, codec, stream);
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_cache_attend(const AttendParams& p, uint32_t codec, uint32_t head_dim, uint32_t tile_rows,
                               hipStream_t stream) {
  switch (head_dim) {
    case 32: return launch_tile<32>(p, codec, tile_rows, stream);
    case 64: return launch_tile<64>(p, codec, tile_rows, stream);
    case 128: return launch_tile<128>(p, codec, tile_rows, stream);
    case 256: return launch_tile<256>(p, codec, tile_rows, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace kvc
