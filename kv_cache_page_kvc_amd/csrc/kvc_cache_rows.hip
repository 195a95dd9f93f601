// kvc_cache_rows.hip -- gfx950 kernels that write rows of K and V into the
// resident 8-bit cache and read them back.
//
// A page of one KV head holds T tokens of K as [token][D] and of V as
// [D][token], 8-bit codes with one FP32 scale a component.  A wave owns one
// (page, head, component) of the call, so nothing is shared between waves: it
// takes the largest |x| of the new tokens, sets the scale, and stores codes.
//  K: a lane takes 8 consecutive dimensions of a token (16 bytes in, 8 out).
//  V: a lane takes 2 dimensions of up to 16 consecutive tokens, so that its
//     codes of one dimension are consecutive bytes: 4-byte loads that
//     together cover whole rows, one store a dimension.
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

template <int D, uint32_t CODEC, int DT>
__global__ __launch_bounds__(256) void cache_write_kernel(RowsParams p) {
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t item = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= (uint64_t)p.units * p.c.heads * 2) return;
  const int comp = (int)(item & 1);
  const uint32_t uh = (uint32_t)(item >> 1), h = uh % p.c.heads;
  const PageWork w = page_work(p, uh / p.c.heads);
  if (w.page < 0) return;
  const int T = 1 << p.c.tshift, p0 = w.page_no * T;
  const RowsView rv = comp ? p.v : p.k;
  // element (position t, dimension 0); positions count from s0
  const uint16_t* src = rv.data + (int64_t)(w.s.r0 + (w.s0 - w.s.start)) * rv.stride_row + (int64_t)h * rv.stride_head;
  uint8_t* codes = (comp ? p.c.v_codes : p.c.k_codes) + w.page * p.c.stride_page + (int64_t)h * T * D;
  float* scale = (comp ? p.c.v_scales : p.c.k_scales) + w.page * p.c.stride_scale + h;
  const int n = w.s1 - w.s0;

  // the largest finite |x| of the new tokens
  constexpr int LPT = D / 8, TPI = 64 / LPT;
  const int lt = (int)lane / LPT, ld = ((int)lane % LPT) * 8;
  uint32_t am = 0, odd = 0;
  for (int t = lt; t < n; t += TPI) {
    const uint4 x = ld_global16(src + (int64_t)t * rv.stride_row + ld);
    const uint32_t a[8] = {x.x & 0x7FFFu, x.x >> 16 & 0x7FFFu, x.y & 0x7FFFu, x.y >> 16 & 0x7FFFu,
                           x.z & 0x7FFFu, x.z >> 16 & 0x7FFFu, x.w & 0x7FFFu, x.w >> 16 & 0x7FFFu};
#pragma unroll
    for (int i = 0; i < 8; i++) {
      const bool fin = a[i] < kNonfinite<DT>;
      am = max(am, fin ? a[i] : 0u);
      odd |= fin ? 0u : 1u;
    }
  }
  am = wave_umax(am);
  if (__any((int)odd)) flag_seq(p.b, w.s.b, KVC_SEQ_NONFINITE);
  const bool fresh = w.s0 == p0;
  const float need = scale_rule<CODEC>(unpack2<DT>(am).x), old = fresh ? 0.0f : *scale;
  const bool usable = old > 0.0f && old < __builtin_inff();    // else nothing was written there
  const float s = usable ? fmaxf(old, need) : need;
  const bool grown = !fresh && s != old;
  const float from = usable ? old : 0.0f;
  if (lane == 0 && (fresh || grown)) *scale = s;

  if (comp == 0) {
    if (grown)
      for (int t = lt; t < w.s0 - p0; t += TPI) {
        uint8_t* at = codes + t * D + ld;
        const uint2 c = ld_global8(at);
        st_global8(at, make_uint2(requant4<CODEC>(c.x, from, s), requant4<CODEC>(c.y, from, s)));
      }
    for (int t = lt; t < n; t += TPI) {
      const uint4 x = ld_global16(src + (int64_t)t * rv.stride_row + ld);
      const f32x2 a = unpack2<DT>(x.x), b = unpack2<DT>(x.y), c = unpack2<DT>(x.z), d = unpack2<DT>(x.w);
      st_global8(codes + (w.s0 - p0 + t) * D + ld, make_uint2(quant4<CODEC>(a.x / s, a.y / s, b.x / s, b.y / s),
                                                              quant4<CODEC>(c.x / s, c.y / s, d.x / s, d.y / s)));
    }
    return;
  }
  using V = VGeo<D>;
  const int q0 = w.s0 - p0, q1 = w.s1 - p0;                    // new tokens of the page
  const int part = V::PARTS == 1 ? 0 : (int)lane / (D / 2);
  for (int g = grown ? 0 : q0 & ~15; g < q1; g += 16)
#pragma unroll
    for (int r = 0; r < V::ROUNDS; r++) {
      const int d = r * 128 + 2 * ((int)lane % (D / 2 < 64 ? D / 2 : 64)), t0 = g + part * V::TOK;
      uint32_t x[V::TOK];
#pragma unroll
      for (int k = 0; k < V::TOK; k++) {
        const int t = t0 + k;
        x[k] = t >= q0 && t < q1 ? ld_global4(src + (int64_t)(t - q0) * rv.stride_row + d) : 0u;
      }
      uint32_t* at[2] = {(uint32_t*)(codes + (int64_t)d * T + t0), (uint32_t*)(codes + (int64_t)(d + 1) * T + t0)};
#pragma unroll
      for (int k = 0; k < V::TOK; k += 4) {
        const f32x2 a = unpack2<DT>(x[k]), b = unpack2<DT>(x[k + 1]), c = unpack2<DT>(x[k + 2]),
                    e = unpack2<DT>(x[k + 3]);
        const uint32_t now[2] = {quant4<CODEC>(a.x / s, b.x / s, c.x / s, e.x / s),
                                 quant4<CODEC>(a.y / s, b.y / s, c.y / s, e.y / s)};
        const uint32_t before = low_bytes(q0 - (t0 + k)), upto = low_bytes(q1 - (t0 + k));
        const uint32_t mine = upto & ~before;
        if (mine == ~0u) {
          at[0][k / 4] = now[0];
          at[1][k / 4] = now[1];
        } else if (mine || (grown && before)) {
#pragma unroll
          for (int i = 0; i < 2; i++) {
            const uint32_t was = at[i][k / 4], kept = grown ? requant4<CODEC>(was, from, s) : was;
            at[i][k / 4] = (now[i] & mine) | (kept & before) | (was & ~(mine | before));
          }
        }
      }
    }
}

template <int D, uint32_t CODEC, int DT>
__global__ __launch_bounds__(256) void cache_read_kernel(RowsParams p) {
  const uint32_t lane = threadIdx.x & 63;
  const uint64_t item = (uint64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (item >= (uint64_t)p.units * p.c.heads * 2) return;
  const int comp = (int)(item & 1);
  const uint32_t uh = (uint32_t)(item >> 1), h = uh % p.c.heads;
  const PageWork w = page_work(p, uh / p.c.heads);
  if (!w.s.ok) return;
  const RowsView rv = comp ? p.v : p.k;
  uint16_t* rows = rv.data + (int64_t)w.s.r0 * rv.stride_row + (int64_t)h * rv.stride_head;
  constexpr int LPT = D / 8, TPI = 64 / LPT;
  const int lt = (int)lane / LPT, ld = ((int)lane % LPT) * 8;
  // rows without a position, and rows whose page is none, are zero
  int z0 = 0, z1 = w.s.unit == 0 ? min(w.s.n, max(-w.s.start, 0)) : 0;
  for (int i = z0 + lt; i < z1; i += TPI) st_global16(rows + (int64_t)i * rv.stride_row + ld, make_uint4(0, 0, 0, 0));
  if (w.s0 >= w.s1) return;
  if (w.page < 0) {
    for (int i = w.s0 - w.s.start + lt; i < w.s1 - w.s.start; i += TPI)
      st_global16(rows + (int64_t)i * rv.stride_row + ld, make_uint4(0, 0, 0, 0));
    return;
  }
  const int T = 1 << p.c.tshift, p0 = w.page_no * T, q0 = w.s0 - p0, q1 = w.s1 - p0;
  uint16_t* dst = rows + (int64_t)(w.s0 - w.s.start) * rv.stride_row;      // of token q0
  const uint8_t* codes = (comp ? p.c.v_codes : p.c.k_codes) + w.page * p.c.stride_page + (int64_t)h * T * D;
  const float s = (comp ? p.c.v_scales : p.c.k_scales)[w.page * p.c.stride_scale + h];
  if (comp == 0) {
    for (int t = q0 + lt; t < q1; t += TPI) {
      const uint2 c = ld_global8(codes + t * D + ld);
      float x[8];
      codes4<CODEC>(c.x, x);
      codes4<CODEC>(c.y, x + 4);
      st_global16(dst + (int64_t)(t - q0) * rv.stride_row + ld,
                  make_uint4(pack2<DT>(x[0] * s, x[1] * s), pack2<DT>(x[2] * s, x[3] * s),
                             pack2<DT>(x[4] * s, x[5] * s), pack2<DT>(x[6] * s, x[7] * s)));
    }
    return;
  }
  using V = VGeo<D>;
  const int part = V::PARTS == 1 ? 0 : (int)lane / (D / 2);
  for (int g = q0 & ~15; g < q1; g += 16)
#pragma unroll
    for (int r = 0; r < V::ROUNDS; r++) {
      const int d = r * 128 + 2 * ((int)lane % (D / 2 < 64 ? D / 2 : 64)), t0 = g + part * V::TOK;
      const uint32_t* at[2] = {(const uint32_t*)(codes + (int64_t)d * T + t0),
                               (const uint32_t*)(codes + (int64_t)(d + 1) * T + t0)};
#pragma unroll
      for (int k = 0; k < V::TOK; k += 4) {
        float a[4], b[4];
        codes4<CODEC>(at[0][k / 4], a);
        codes4<CODEC>(at[1][k / 4], b);
#pragma unroll
        for (int i = 0; i < 4; i++) {
          const int t = t0 + k + i;
          if (t >= q0 && t < q1)
            *(g_u32*)(dst + (int64_t)(t - q0) * rv.stride_row + d) = pack2<DT>(a[i] * s, b[i] * s);
        }
      }
    }
}

template <bool WRITE, int D, uint32_t CODEC>
hipError_t launch_dt(const RowsParams& p, uint32_t dtype, hipStream_t stream) {
  const uint64_t items = (uint64_t)p.units * p.c.heads * 2;
  const dim3 grid((uint32_t)((items + 3) / 4));
  if constexpr (WRITE) {
    if (dtype == KVC_BF16) cache_write_kernel<D, CODEC, KVC_BF16><<<grid, 256, 0, stream>>>(p);
    else cache_write_kernel<D, CODEC, KVC_FP16><<<grid, 256, 0, stream>>>(p);
  } else {
    if (dtype == KVC_BF16) cache_read_kernel<D, CODEC, KVC_BF16><<<grid, 256, 0, stream>>>(p);
    else cache_read_kernel<D, CODEC, KVC_FP16><<<grid, 256, 0, stream>>>(p);
  }
  return hipGetLastError();
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
