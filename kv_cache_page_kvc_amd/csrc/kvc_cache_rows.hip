// kvc_cache_rows.hip -- gfx950 kernels that write rows of K and V into the
// resident 8-bit cache and read them back.
//
// A page of one KV head holds T tokens of K as [token][D] and of V as
// [D][token], 8-bit codes with one FP32 scale a component.  A wave takes 16
// tokens of one (page, head, component); in a write the waves of a larger page
// share its largest |x| through LDS, then each stores its tokens' codes from
// the registers that hold the rows.
//  K: a lane takes 8 consecutive dimensions of a token (16 bytes in, 8 out).
//  V: a lane takes 2 dimensions of up to 16 consecutive tokens, so that its
//     codes of one dimension are consecutive bytes: 4-byte loads that
//     together cover whole rows, one store a dimension.
#include <type_traits>

#include "kvc_cache_device.h"

namespace kvc {
namespace {

// A lane's share of V in a group of 16 tokens: PARTS lanes split the tokens
// of a dimension pair, each with TOK tokens; ROUNDS passes cover D.
template <int D>
struct VGeo {
  static constexpr int PARTS = D >= 128 ? 1 : 128 / D;
  static constexpr int TOK = 16 / PARTS;
  static constexpr int ROUNDS = D >= 128 ? D / 128 : 1;
};

// the page of a unit: page number in the sequence, positions [s0, s1) of the call in it
struct PageWork {
  Seq s;
  int page_no, s0, s1;
  int64_t page;          // id; < 0: none
};
__device__ __forceinline__ PageWork page_work(const RowsParams& p, uint32_t unit) {
  PageWork w;
  w.s = seq_of_unit(p.b, unit);
  w.page = -1;
  w.s0 = w.s1 = 0;
  if (!w.s.ok) return w;
  const int T = 1 << p.c.tshift;
  const int first = max(w.s.start, 0);
  // 64 bits: a unit beyond the sequence's pages may lie past 2^31 positions
  const int64_t no = (int64_t)(first >> p.c.tshift) + w.s.unit;
  if (no * T >= w.s.len || w.s.n == 0) return w;
  w.page_no = (int)no;
  w.s0 = max(first, w.page_no * T);
  w.s1 = min(w.s.len, w.page_no * T + T);
  const int32_t id = p.b.table[(int64_t)w.s.b * p.b.stride_table + w.page_no];
  if (id < 0 || (uint32_t)id >= p.c.num_pages) flag_seq(p.b, w.s.b, KVC_SEQ_BAD_PAGE);
  else w.page = id;
  return w;
}

template <uint32_t CODEC>
__device__ __forceinline__ float scale_rule(float amax) {
  const float a = fmaxf(amax, 1e-12f);
  return CODEC == C_FP8 ? a * (1.0f / 448.0f) : a / 127.0f;
}
template <uint32_t CODEC>
__device__ __forceinline__ uint32_t requant4(uint32_t w, float from, float to) {
  float x[4];
  codes4<CODEC>(w, x);
  return quant4<CODEC>(x[0] * from / to, x[1] * from / to, x[2] * from / to, x[3] * from / to);
}
// bytes [0, n) of a dword
__device__ __forceinline__ uint32_t low_bytes(int n) { return n <= 0 ? 0u : (n >= 4 ? ~0u : (1u << (8 * n)) - 1u); }

// Codes of four values x, y in packed pairs against scale s (r = 1 / s).
// EXACT: the IEEE quotient, any x.  Else x / s from r and one FMA residual step,
// for finite |x| at most the amax that s was formed from: the code is the IEEE
// quotient's (the same sequence and claim as the page codecs', checked there
// over every such pair), and needs no clipping -- the largest quotient rounds
// to the largest code.
template <uint32_t CODEC, bool EXACT>
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d, float s, float r) {
  if constexpr (EXACT) {
    return quant4<CODEC>(a / s, b / s, c / s, d / s);
  } else {
    float q[4] = {a, b, c, d};
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const float x = q[i], q0 = x * r;
      q[i] = fmaf(fmaf(-q0, s, x), r, q0);
      if constexpr (CODEC == C_FP8) q[i] = copysignf(q[i], x);   // the residual step turns -0 into 0
    }
    if constexpr (CODEC == C_FP8) {
      const int lo = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
      return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], lo, true);
    } else {
      // RNE(q) in the low byte of q + 1.5 * 2^23
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; i++) u[i] = __float_as_uint(q[i] + 12582912.0f);
      return __builtin_amdgcn_perm(__builtin_amdgcn_perm(u[3], u[2], 0x0C0C0400u),
                                   __builtin_amdgcn_perm(u[1], u[0], 0x0C0C0400u), 0x05040100u);
    }
  }
}

// |x| of a packed pair as integers; not finite ones count as 0 and set odd
template <int DT>
__device__ __forceinline__ void pair_max(uint32_t w, uint32_t& am, uint32_t& odd) {
  const uint32_t a = w & 0x7FFFu, b = w >> 16 & 0x7FFFu;
  const bool fa = a < kNonfinite<DT>, fb = b < kNonfinite<DT>;
  am = max(am, max(fa ? a : 0u, fb ? b : 0u));
  odd |= fa && fb ? 0u : 1u;
}

// Waves of an item (page, head, component), and its groups of 16 tokens a wave.
// A row is read once and stays in registers between its maximum and its codes,
// so a write moves what it must: 64K tokens of 8 heads of 128 (403 MB in and
// out) take 82 us, 4.9 TB/s, where a copy reaches 5.0; with the rows read twice
// it was 124.  Small calls are bound by the chain cu_rows -> block table -> rows
// -> scale: one token 4.8 us, 256 users' tokens 8.5.  At D = 64 a token's head
// is 128 bytes, and 24 ragged prompts (116 MB) reach 3.0 TB/s, 38.6 us.
constexpr int item_waves(int T) { return T >= 128 ? 8 : T / 16; }

template <int D, uint32_t CODEC, int DT, int T>
__global__ __launch_bounds__(item_waves(T) == 8 ? 512 : 256) void cache_write_kernel(RowsParams p) {
  constexpr int WPI = item_waves(T), GPW = T / 16 / WPI, WAVES = WPI == 8 ? 8 : 4;
  constexpr int LPT = D / 8, TPI = 64 / LPT, KL = 16 / TPI;      // K: lanes a token, tokens a load, loads a group
  using V = VGeo<D>;
  constexpr int REGS = GPW * (4 * KL > V::ROUNDS * V::TOK ? 4 * KL : V::ROUNDS * V::TOK);
  __shared__ uint32_t s_max[WAVES], s_odd[WAVES];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6), sub = wave % WPI;
  const uint64_t item = (uint64_t)blockIdx.x * (WAVES / WPI) + wave / WPI, items = (uint64_t)p.units * p.c.heads * 2;
  const uint32_t h = (uint32_t)(item % p.c.heads), uc = (uint32_t)(item / p.c.heads);
  const int comp = (int)(uc & 1);
  PageWork w;
  w.page = -1;
  if (item < items) w = page_work(p, uc >> 1);
  const bool work = w.page >= 0;
  if (WPI == 1 && !work) return;
  if (!work) w.s0 = w.s1 = w.page_no = 0;
  const int p0 = w.page_no * T, q0 = w.s0 - p0, q1 = w.s1 - p0;  // new tokens of the page
  const RowsView rv = comp ? p.v : p.k;
  // element (first new token, dimension 0)
  const uint16_t* src = rv.data + (work ? (int64_t)(w.s.r0 + (w.s0 - w.s.start)) * rv.stride_row + (int64_t)h * rv.stride_head : 0);
  uint8_t* codes = (comp ? p.c.v_codes : p.c.k_codes) + (work ? w.page * p.c.stride_page + (int64_t)h * T * D : 0);
  float* scale = (comp ? p.c.v_scales : p.c.k_scales) + (work ? w.page * p.c.stride_scale + h : 0);
  const int lt = lane / LPT, ld = (lane % LPT) * 8;
  const int part = V::PARTS == 1 ? 0 : lane / (D / 2), vd = 2 * (lane % (D / 2 < 64 ? D / 2 : 64));

  const bool fresh = q0 == 0;
  const float old = fresh || !work ? 0.0f : *scale;            // before any wave sets it, below
  // the rows, into registers, and V's codes beside them where a lane's tokens are not all new
  uint32_t x[REGS], was[GPW * V::ROUNDS * 2 * (V::TOK / 4)];
  uint32_t am = 0, odd = 0;
#pragma unroll
  for (int k = 0; k < GPW; k++) {
    const int t0 = 16 * (sub + WPI * k);
    if (t0 >= q1 || t0 + 16 <= q0) continue;
    if (comp == 0) {
#pragma unroll
      for (int i = 0; i < KL; i++) {
        const int t = t0 + lt + TPI * i;
        const uint4 v = t >= q0 && t < q1 ? ld_global16(src + (int64_t)(t - q0) * rv.stride_row + ld) : make_uint4(0, 0, 0, 0);
        uint32_t* at = x + 4 * (k * KL + i);
        at[0] = v.x, at[1] = v.y, at[2] = v.z, at[3] = v.w;
      }
#pragma unroll
      for (int i = 0; i < 4 * KL; i++) pair_max<DT>(x[4 * k * KL + i], am, odd);
    } else {
#pragma unroll
      for (int i = 0; i < V::ROUNDS * V::TOK; i++) {
        const int t = t0 + part * V::TOK + i % V::TOK, d = vd + 128 * (i / V::TOK);
        x[k * V::ROUNDS * V::TOK + i] = t >= q0 && t < q1 ? ld_global4(src + (int64_t)(t - q0) * rv.stride_row + d) : 0u;
      }
      const int tl = t0 + part * V::TOK;
      if (tl < q0 || tl + V::TOK > q1)
#pragma unroll
        for (int i = 0; i < V::ROUNDS * 2; i++) {
          const uint8_t* at = codes + (int64_t)(vd + 128 * (i / 2) + i % 2) * T + tl;
#pragma unroll
          for (int j = 0; j < V::TOK / 4; j++) was[(k * V::ROUNDS * 2 + i) * (V::TOK / 4) + j] = ld_global4(at + 4 * j);
        }
#pragma unroll
      for (int i = 0; i < V::ROUNDS * V::TOK; i++) pair_max<DT>(x[k * V::ROUNDS * V::TOK + i], am, odd);
    }
  }
  am = wave_umax(am);
  odd = __any((int)odd) ? 1u : 0u;
  if constexpr (WPI > 1) {
    if (lane == 0) {
      s_max[wave] = am;
      s_odd[wave] = odd;
    }
    __syncthreads();
    const int first = wave - sub;
#pragma unroll
    for (int i = 0; i < WPI; i++) {
      am = max(am, s_max[first + i]);
      odd |= s_odd[first + i];
    }
    if (!work) return;
  }
  if (odd && sub == 0) flag_seq(p.b, w.s.b, KVC_SEQ_NONFINITE);

  const float need = scale_rule<CODEC>(unpack2<DT>(am).x);
  const bool usable = old > 0.0f && old < __builtin_inff();    // else nothing was written there
  const float s = usable ? fmaxf(old, need) : need;
  const bool grown = !fresh && s != old;
  const float from = usable ? old : 0.0f, r = 1.0f / s;
  if (lane == 0 && sub == 0 && (fresh || grown)) *scale = s;

  auto store = [&](auto exact) {
    constexpr bool EXACT = decltype(exact)::value;
#pragma unroll
    for (int k = 0; k < GPW; k++) {
      const int t0 = 16 * (sub + WPI * k);
      const bool some = t0 < q1 && t0 + 16 > q0;
      if (comp == 0) {
        if (some)
#pragma unroll
          for (int i = 0; i < KL; i++) {
            const int t = t0 + lt + TPI * i;
            const uint32_t* at = x + 4 * (k * KL + i);
            const f32x2 a = unpack2<DT>(at[0]), b = unpack2<DT>(at[1]), c = unpack2<DT>(at[2]), d = unpack2<DT>(at[3]);
            if (t >= q0 && t < q1)
              st_global8(codes + t * D + ld, make_uint2(codes_of<CODEC, EXACT>(a.x, a.y, b.x, b.y, s, r),
                                                        codes_of<CODEC, EXACT>(c.x, c.y, d.x, d.y, s, r)));
          }
        if (EXACT && grown)
          for (int t = t0 + lt; t < min(q0, t0 + 16); t += TPI) {
            uint8_t* at = codes + t * D + ld;
            const uint2 c = ld_global8(at);
            st_global8(at, make_uint2(requant4<CODEC>(c.x, from, s), requant4<CODEC>(c.y, from, s)));
          }
      } else if (some || (EXACT && grown && t0 < q0)) {
        const int tl = t0 + part * V::TOK;
#pragma unroll
        for (int rd = 0; rd < V::ROUNDS; rd++) {
          const uint32_t* xv = x + (k * V::ROUNDS + rd) * V::TOK;
          uint32_t now[2][V::TOK / 4];
#pragma unroll
          for (int j = 0; j < V::TOK; j += 4) {
            now[0][j / 4] = now[1][j / 4] = 0;
            if (EXACT && (tl + j + 4 <= q0 || tl + j >= q1)) continue;   // divisions are slow, and single tokens common
            f32x2 y[4];
#pragma unroll
            for (int i = 0; i < 4; i++) y[i] = unpack2<DT>(some ? xv[j + i] : 0u);
            now[0][j / 4] = codes_of<CODEC, EXACT>(y[0].x, y[1].x, y[2].x, y[3].x, s, r);
            now[1][j / 4] = codes_of<CODEC, EXACT>(y[0].y, y[1].y, y[2].y, y[3].y, s, r);
          }
#pragma unroll
          for (int i = 0; i < 2; i++) {
            uint32_t* at = (uint32_t*)(codes + (int64_t)(vd + 128 * rd + i) * T + tl);
            if (tl >= q0 && tl + V::TOK <= q1) {
              if constexpr (V::TOK == 16) st_global16(at, make_uint4(now[i][0], now[i][1], now[i][2], now[i][3]));
              else if constexpr (V::TOK == 8) st_global8(at, make_uint2(now[i][0], now[i][1]));
              else *(g_u32*)at = now[i][0];
            } else {
#pragma unroll
              for (int j = 0; j < V::TOK / 4; j++) {
                const uint32_t before = low_bytes(q0 - (tl + 4 * j)), upto = low_bytes(q1 - (tl + 4 * j));
                const uint32_t mine = upto & ~before;
                if (mine || (EXACT && grown && before)) {
                  const uint32_t then = some ? was[((k * V::ROUNDS + rd) * 2 + i) * (V::TOK / 4) + j] : ld_global4(at + j);
                  const uint32_t kept = EXACT && grown ? requant4<CODEC>(then, from, s) : then;
                  *(g_u32*)(at + j) = (now[i][j] & mine) | (kept & before) | (then & ~(mine | before));
                }
              }
            }
          }
        }
      }
    }
  };
  // a page's first scale comes from these rows; an older one, or values that
  // are not finite, take the IEEE division
  if (fresh && !odd) store(std::false_type{});
  else store(std::true_type{});
}

// A wave reads 16 tokens of one (page, head, component): 64K tokens of 8 heads
// of 128 take 88 us, 4.6 TB/s, bound by HBM.
template <int D, uint32_t CODEC, int DT, int T>
__global__ __launch_bounds__(256) void cache_read_kernel(RowsParams p) {
  constexpr int GROUPS = T / 16;
  const int lane = threadIdx.x & 63;
  const uint64_t id = (uint64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const uint64_t item = id / GROUPS;
  const int t0 = 16 * (int)(id % GROUPS);
  if (item >= (uint64_t)p.units * p.c.heads * 2) return;
  const uint32_t h = (uint32_t)(item % p.c.heads), uc = (uint32_t)(item / p.c.heads);
  const int comp = (int)(uc & 1);
  const PageWork w = page_work(p, uc >> 1);
  if (!w.s.ok) return;
  const RowsView rv = comp ? p.v : p.k;
  uint16_t* rows = rv.data + (int64_t)w.s.r0 * rv.stride_row + (int64_t)h * rv.stride_head;
  constexpr int LPT = D / 8, TPI = 64 / LPT, KL = 16 / TPI;
  const int lt = lane / LPT, ld = (lane % LPT) * 8;
  // rows without a position, and rows whose page is none, are zero
  if (w.s.unit == 0 && t0 == 0)
    for (int i = lt; i < min(w.s.n, max(-w.s.start, 0)); i += TPI)
      st_global16(rows + (int64_t)i * rv.stride_row + ld, make_uint4(0, 0, 0, 0));
  if (w.s0 >= w.s1) return;
  const int p0 = w.page_no * T, q0 = max(w.s0 - p0, t0), q1 = min(w.s1 - p0, t0 + 16);
  if (q0 >= q1) return;
  uint16_t* dst = rows + (int64_t)(p0 - w.s.start) * rv.stride_row;        // of the page's first token
  if (w.page < 0) {
    for (int t = q0 + lt; t < q1; t += TPI) st_global16(dst + (int64_t)t * rv.stride_row + ld, make_uint4(0, 0, 0, 0));
    return;
  }
  const uint8_t* codes = (comp ? p.c.v_codes : p.c.k_codes) + w.page * p.c.stride_page + (int64_t)h * T * D;
  const float s = (comp ? p.c.v_scales : p.c.k_scales)[w.page * p.c.stride_scale + h];
  if (comp == 0) {
    uint2 c[KL];
#pragma unroll
    for (int i = 0; i < KL; i++) c[i] = ld_global8(codes + (t0 + lt + TPI * i) * D + ld);
#pragma unroll
    for (int i = 0; i < KL; i++) {
      const int t = t0 + lt + TPI * i;
      float x[8];
      codes4<CODEC>(c[i].x, x);
      codes4<CODEC>(c[i].y, x + 4);
      if (t >= q0 && t < q1)
        st_global16(dst + (int64_t)t * rv.stride_row + ld,
                    make_uint4(pack2<DT>(x[0] * s, x[1] * s), pack2<DT>(x[2] * s, x[3] * s),
                               pack2<DT>(x[4] * s, x[5] * s), pack2<DT>(x[6] * s, x[7] * s)));
    }
    return;
  }
  using V = VGeo<D>;
  const int part = V::PARTS == 1 ? 0 : lane / (D / 2), vd = 2 * (lane % (D / 2 < 64 ? D / 2 : 64));
  const int tl = t0 + part * V::TOK;
  uint32_t c[V::ROUNDS][2][V::TOK / 4];
#pragma unroll
  for (int r = 0; r < V::ROUNDS; r++)
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const uint8_t* at = codes + (int64_t)(vd + 128 * r + i) * T + tl;
      if constexpr (V::TOK == 16) {
        const uint4 v = ld_global16(at);
        c[r][i][0] = v.x, c[r][i][1] = v.y, c[r][i][2] = v.z, c[r][i][3] = v.w;
      } else if constexpr (V::TOK == 8) {
        const uint2 v = ld_global8(at);
        c[r][i][0] = v.x, c[r][i][1] = v.y;
      } else {
        c[r][i][0] = ld_global4(at);
      }
    }
#pragma unroll
  for (int r = 0; r < V::ROUNDS; r++)
#pragma unroll
    for (int j = 0; j < V::TOK; j += 4) {
      float a[4], b[4];
      codes4<CODEC>(c[r][0][j / 4], a);
      codes4<CODEC>(c[r][1][j / 4], b);
#pragma unroll
      for (int i = 0; i < 4; i++) {
        const int t = tl + j + i;
        if (t >= q0 && t < q1)
          *(g_u32*)(dst + (int64_t)t * rv.stride_row + vd + 128 * r) = pack2<DT>(a[i] * s, b[i] * s);
      }
    }
}

template <bool WRITE, int D, uint32_t CODEC, int DT>
hipError_t launch_page(const RowsParams& p, hipStream_t stream) {
  const uint64_t items = (uint64_t)p.units * p.c.heads * 2;
  auto go = [&](auto tokens) {
    constexpr int T = decltype(tokens)::value, WPI = item_waves(T), IPB = WPI >= 4 ? 1 : 4 / WPI;
    if constexpr (WRITE)
      cache_write_kernel<D, CODEC, DT, T>
          <<<(uint32_t)((items + IPB - 1) / IPB), WPI == 8 ? 512 : 256, 0, stream>>>(p);
    else
      cache_read_kernel<D, CODEC, DT, T><<<(uint32_t)((items * (T / 16) + 3) / 4), 256, 0, stream>>>(p);
    return hipGetLastError();
  };
  switch (1 << p.c.tshift) {
    case 16: return go(std::integral_constant<int, 16>{});
    case 32: return go(std::integral_constant<int, 32>{});
    case 64: return go(std::integral_constant<int, 64>{});
    case 128: return go(std::integral_constant<int, 128>{});
    case 256: return go(std::integral_constant<int, 256>{});
  }
  return hipErrorInvalidValue;
}
template <bool WRITE, int D, uint32_t CODEC>
hipError_t launch_dt(const RowsParams& p, uint32_t dtype, hipStream_t stream) {
  return dtype == KVC_BF16 ? launch_page<WRITE, D, CODEC, KVC_BF16>(p, stream)
                           : launch_page<WRITE, D, CODEC, KVC_FP16>(p, stream);
}
template <bool WRITE, int D>
hipError_t launch_codec(const RowsParams& p, uint32_t codec, uint32_t dtype, hipStream_t stream) {
  return codec == C_FP8 ? launch_dt<WRITE, D, C_FP8>(p, dtype, stream) : launch_dt<WRITE, D, C_INT8>(p, dtype, stream);
}
template <bool WRITE>
hipError_t launch_rows(const RowsParams& p, uint32_t codec, uint32_t dtype, uint32_t d, hipStream_t stream) {
  switch (d) {
    case 32: return launch_codec<WRITE, 32>(p, codec, dtype, stream);
    case 64: return launch_codec<WRITE, 64>(p, codec, dtype, stream);
    case 128: return launch_codec<WRITE, 128>(p, codec, dtype, stream);
    case 256: return launch_codec<WRITE, 256>(p, codec, dtype, stream);
  }
  return hipErrorInvalidValue;
}

}  // namespace

hipError_t launch_cache_write(const RowsParams& p, uint32_t codec, uint32_t dtype, uint32_t head_dim,
                              hipStream_t stream) {
  return launch_rows<true>(p, codec, dtype, head_dim, stream);
}
hipError_t launch_cache_read(const RowsParams& p, uint32_t codec, uint32_t dtype, uint32_t head_dim,
                             hipStream_t stream) {
  return launch_rows<false>(p, codec, dtype, head_dim, stream);
}

}  // namespace kvc
