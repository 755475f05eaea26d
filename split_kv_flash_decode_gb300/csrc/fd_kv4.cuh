// Decode over a 4-bit cache: the per-warp mma.sync consumer, and the stream kernel that runs by
// default.  Included by fd_kernel.cuh, which provides the primitives.
#pragma once

#include <cfloat>

namespace fd {
namespace dev {

// D = A * B for one m16n8k16 f16 tile.
__device__ __forceinline__ void mma16816_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%10,%10,%10,%10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// One warp's share of the attention of one (sequence, KV head): running (m, l, O^T) of its G
// query heads over the 16-token blocks it is given.
//
// S = K q^T and O^T += V^T P^T on mma.sync m16n8k16 with tokens (then head dimensions) on M and
// the heads on N.  Index permutations make each thread's fragment bytes contiguous: thread quad t
// covers elements t D/4 + 4 kk + {0, 1} (a0/a1/b0) and + {2, 3} (a2/a3/b1) in k-step kk of S; row
// g / g + 8 of m-tile mi of O^T is dim g D/8 + 2 mi / + 1.  An element is E2M1 value x E4M3
// scale, at most 6 significant bits and 2^-10 .. 2688 in size: exact in f16, so both products run
// on f16 mma whatever q's type.  bf16 q is brought to f16 range by a power of two per head (its 8
// significant bits stay; elements below 2^-14 of the head's largest lose at most 2^-25 of it, the
// size of fp32's own rounding).
//
// The E2M1 conversion is one instruction per pair at half rate, the scale one more at full rate.
// (Measured per 8 values of a warp: 8 cycles for the four conversions, 10 for an integer format
// by mask-and-or, 24 for E2M1 by masks and shifts.)
//
// Groups of up to 4 heads leave half of N = 8 empty.  The empty columns take the same heads
// again, with the rounding residuals of their weights: P.V then sees hi + lo, 22 significant
// bits, for the same number of mma.  Larger groups round the weights once (11 bits, as decodes over
// an f16 or E4M3 cache do); lr sums the rounded weights, which also normalise the output.  That is a
// choice: a second set of mma for the residuals takes 64 sequences of 8K tokens from 97.2 to 109.4 us
// (G = 8) and from 142.5 to 164.1 (G = 16), and 128K tokens from 32.0 to 35.4 (G = 8), to bring the
// relative error of an f16 output from 2.9e-4 to the 2.1e-4 of its own rounding.
template <typename T, int D, int G>
struct Kv4Warp {
  static constexpr int KT = D / 16;               // k-steps of S, m-tiles of O^T
  static constexpr int NT = G >= 8 ? G / 8 : 1;   // N tiles of 8 columns
  static constexpr int NW = D / 64;               // K words of 8 elements per thread and row, x 2
  static constexpr int BLK = 16 * ring_row_bytes(kPathMmaKv4, D);  // bytes between blocks in the ring
  static constexpr bool kTwice = G <= 4;          // columns 4 .. 7: heads 0 .. 3 again (residuals)
  static_assert(BLK % 128 == 0, "every block can be the destination of a TMA box");

  uint32_t qb[NT][KT][2];
  float scA[NT], scB[NT];  // log2-domain logit scales of this thread's two columns
  float o[NT][KT][4];
  // l: sums of the fp32 weights (for lse); lr: of the weights P.V uses (for out).
  float mA[NT], mB[NT], lA[NT], lB[NT], lrA[NT], lrB[NT];

  // q of (sequence, KV head) as it is stored: issues the loads.  (All warps read all of it, 16 lines
  // per load: 8-byte loads took 0.6 us more at G = 16.)
  __device__ __forceinline__ void fetch_q(const Params& p, int b, int kvh) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int head = kTwice ? g & 3 : nt * 8 + g;
      const bool real = head < G;
      const uint4* qh = reinterpret_cast<const uint4*>(
          reinterpret_cast<const T*>(p.q) + ((int64_t)b * p.Hq + kvh * G + (real ? head : 0)) * D +
          t * (D / 4));
#pragma unroll
      for (int kk = 0; kk < KT; kk += 2) {
        const uint4 x = real ? qh[kk / 2] : make_uint4(0u, 0u, 0u, 0u);
        qb[nt][kk][0] = x.x;
        qb[nt][kk][1] = x.y;
        qb[nt][kk + 1][0] = x.z;
        qb[nt][kk + 1][1] = x.w;
      }
    }
  }
  // The empty state.  Its maximum is the lowest finite value: -inf logits (products that overflow)
  // then have the weight 0 also where a warp has met no other, while -inf - -inf would be NaN.
  __device__ __forceinline__ void reset() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int mi = 0; mi < KT; ++mi) o[nt][mi][0] = o[nt][mi][1] = o[nt][mi][2] = o[nt][mi][3] = 0.f;
      mA[nt] = mB[nt] = -FLT_MAX;
      lA[nt] = lB[nt] = lrA[nt] = lrB[nt] = 0.f;
    }
  }
  // Makes the fetched q the B operand, and starts from the empty state.
  __device__ __forceinline__ void start(const Params& p) {
    const int t = threadIdx.x & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float scale = p.scale_log2;
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        float mx = 0.f;
#pragma unroll
        for (int kk = 0; kk < 2 * KT; ++kk) {
          const float2 f = Elem<T>::to_f2(qb[nt][kk >> 1][kk & 1]);
          mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // Exponent of the largest |q|, kept where 2^e and 2^-e are normal; infinite q: 0.
        int e = (int)(__float_as_uint(mx) >> 23) - 127;
        e = e == 128 ? 0 : max(-126, min(126, e));
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int kk = 0; kk < 2 * KT; ++kk) {
          const float2 f = Elem<T>::to_f2(qb[nt][kk >> 1][kk & 1]);
          qb[nt][kk >> 1][kk & 1] = pack2<__half>(f.x * down, f.y * down);
        }
        scale *= __uint_as_float((uint32_t)(127 + e) << 23);
      }
      scA[nt] = __shfl_sync(0xffffffffu, scale, 8 * t);      // column 2t is lane group g = 2t
      scB[nt] = __shfl_sync(0xffffffffu, scale, 8 * t + 4);
    }
    reset();
  }
  __device__ __forceinline__ void load_q(const Params& p, int b, int kvh) {
    fetch_q(p, b, kvh);
    start(p);
  }

  // SUB blocks of 16 tokens, BLK bytes apart, of which `ntok` (at least one) tokens are valid.
  // Their K loads, conversions and score mma are independent chains, and one max update covers
  // all of them.
  template <int SUB>
  __device__ __forceinline__ void blocks(const uint8_t* kblk, const uint8_t* vblk, int ntok) {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
    // This thread's byte offsets in a block (fd.h, "4-bit blocks").
    const int k_at = g * (D / 2) + t * (D / 8), ks_at = 8 * D + g * (D / 16) + t * (D / 64);
    const int vswap = ((D == 128 ? g : g >> 1) & 1) << 2;
    const int v_at0 = g * D + (t ^ vswap) * (D / 8), v_at1 = g * D + ((t + 4) ^ vswap) * (D / 8);
    const int vs_at = 8 * D + (D == 128 ? g : g >> 1) * 16 + 2 * t;
    float sc[SUB][NT][4];
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      // K: rows g and g + 8 of block u; kw words of 8 elements, ks the scales as pairs.
      uint32_t kw[2][2 * NW], ks[2][NW];
#pragma unroll
      for (int rh = 0; rh < 2; ++rh) {
        const uint8_t* row = kblk + u * BLK + rh * (4 * D) + k_at;
        const uint8_t* srow = kblk + u * BLK + rh * (D / 2) + ks_at;
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(row);
          kw[rh][0] = x.x; kw[rh][1] = x.y; kw[rh][2] = x.z; kw[rh][3] = x.w;
          const uint32_t z = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(srow));
          ks[rh][0] = __byte_perm(z, z, 0x1010);
          ks[rh][1] = __byte_perm(z, z, 0x3232);
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(row);
          kw[rh][0] = x.x; kw[rh][1] = x.y;
          const uint32_t z = e4m3x2_to_f16x2(*srow);
          ks[rh][0] = __byte_perm(z, z, 0x1010);
        }
      }
      // Two accumulators (even and odd k-steps) halve the chains of dependent mma.
      float sd[NT][4];
#pragma unroll
      for (int wi = 0; wi < 2 * NW; ++wi) {  // a word: k-steps 2 wi and 2 wi + 1
        uint32_t x0[4], x1[4];
        e2m1x8_to_f16x8(kw[0][wi], x0);
        e2m1x8_to_f16x8(kw[1][wi], x1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t a[4] = {hmul2(x0[2 * h], ks[0][wi >> 1]), hmul2(x1[2 * h], ks[1][wi >> 1]),
                                 hmul2(x0[2 * h + 1], ks[0][wi >> 1]), hmul2(x1[2 * h + 1], ks[1][wi >> 1])};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            if (wi == 0)
              mma16816_zero(h ? sd[nt] : sc[u][nt], a, qb[nt][h][0], qb[nt][h][1]);
            else
              mma16816<__half>(h ? sd[nt] : sc[u][nt], a, qb[nt][2 * wi + h][0], qb[nt][2 * wi + h][1]);
          }
        }
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[u][nt][i] += sd[nt][i];
    }
    const bool whole = ntok >= 16 * SUB;
    uint32_t pb0[SUB][NT], pb1[SUB][NT];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      float xA = -INFINITY, xB = -INFINITY;
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        // Scaled on its own, not in an fma with the maximum: among logits of 1e30 the unrounded
        // product is far from the rounded maximum, and its exp2 infinite.
        sc[u][nt][0] *= scA[nt];
        sc[u][nt][1] *= scB[nt];
        sc[u][nt][2] *= scA[nt];
        sc[u][nt][3] *= scB[nt];
        if (!whole) {  // tokens past the end are selected away: their bytes may be anything
          if (16 * u + g >= ntok) sc[u][nt][0] = sc[u][nt][1] = -INFINITY;
          if (16 * u + g + 8 >= ntok) sc[u][nt][2] = sc[u][nt][3] = -INFINITY;
        }
        xA = fmaxf(xA, fmaxf(sc[u][nt][0], sc[u][nt][2]));
        xB = fmaxf(xB, fmaxf(sc[u][nt][1], sc[u][nt][3]));
      }
      // Lazy rescale: the maxima are reduced over the column's lanes only when some logit of the
      // warp passes its running maximum by 2^8 (always in a piece's first blocks).
      if (__any_sync(0xffffffffu, xA > mA[nt] + kRescaleThreshold || xB > mB[nt] + kRescaleThreshold)) {
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) {
          xA = fmaxf(xA, __shfl_xor_sync(0xffffffffu, xA, off));
          xB = fmaxf(xB, __shfl_xor_sync(0xffffffffu, xB, off));
        }
        if (xA > mA[nt]) {
          const float corr = ex2(mA[nt] - xA);
          lA[nt] *= corr;
          lrA[nt] *= corr;
#pragma unroll
          for (int mi = 0; mi < KT; ++mi) { o[nt][mi][0] *= corr; o[nt][mi][2] *= corr; }
          mA[nt] = xA;
        }
        if (xB > mB[nt]) {
          const float corr = ex2(mB[nt] - xB);
          lB[nt] *= corr;
          lrB[nt] *= corr;
#pragma unroll
          for (int mi = 0; mi < KT; ++mi) { o[nt][mi][1] *= corr; o[nt][mi][3] *= corr; }
          mB[nt] = xB;
        }
      }
#pragma unroll
      for (int u = 0; u < SUB; ++u) {
        const float pA0 = ex2(sc[u][nt][0] - mA[nt]), pB0 = ex2(sc[u][nt][1] - mB[nt]);
        const float pA1 = ex2(sc[u][nt][2] - mA[nt]), pB1 = ex2(sc[u][nt][3] - mB[nt]);
        lA[nt] += pA0 + pA1;
        lB[nt] += pB0 + pB1;
        uint32_t r0 = pack2<__half>(pA0, pB0), r1 = pack2<__half>(pA1, pB1);
        const float2 w0 = Elem<__half>::to_f2(r0), w1 = Elem<__half>::to_f2(r1);
        if constexpr (kTwice) {
          const float lo = t < 2 ? 0.f : -1.f;  // columns 4 .. 7 keep what the rounding dropped
          r0 = pack2<__half>(fmaf(w0.x, lo, pA0), fmaf(w0.y, lo, pB0));
          r1 = pack2<__half>(fmaf(w1.x, lo, pA1), fmaf(w1.y, lo, pB1));
        } else {
          lrA[nt] += w0.x + w1.x;
          lrB[nt] += w0.y + w1.y;
        }
        // P (tokens x heads, accumulator layout) -> P^T as the B operand (k = token).
        pb0[u][nt] = movmatrix_trans(r0);
        pb1[u][nt] = movmatrix_trans(r1);
      }
    }
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      // V^T: tokens 2t, 2t + 1 (words ve[0], vo[0], scales vs[0]) and 2t + 8, 2t + 9.
      uint32_t ve[2][NW], vo[2][NW], vs[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint8_t* at = vblk + u * BLK + (i ? v_at1 : v_at0);
        if constexpr (D == 128) {
          const uint4 x = *reinterpret_cast<const uint4*>(at);
          ve[i][0] = x.x; ve[i][1] = x.y; vo[i][0] = x.z; vo[i][1] = x.w;
        } else {
          const uint2 x = *reinterpret_cast<const uint2*>(at);
          ve[i][0] = x.x; vo[i][0] = x.y;
        }
        vs[i] = e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(vblk + u * BLK + vs_at + 8 * i));
        if (!whole) {
          // A weight of 0 times a NaN scale would be NaN: scales past the end become 0.
          const int left = ntok - (16 * u + 8 * i + 2 * t);
          if (left < 2) vs[i] = left < 1 ? 0u : vs[i] & 0xffffu;
        }
      }
#pragma unroll
      for (int wi = 0; wi < NW; ++wi) {
        // Half-bytes of the two tokens of a pair side by side: even dims in f[.][0], odd in f[.][1].
        uint32_t f[2][2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t a = ve[i][wi], b = vo[i][wi];
          e2m1x8_to_f16x8((a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u), f[i][0]);
          e2m1x8_to_f16x8(((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u), f[i][1]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t a[4] = {hmul2(f[0][0][j], vs[0]), hmul2(f[0][1][j], vs[0]),
                                 hmul2(f[1][0][j], vs[1]), hmul2(f[1][1][j], vs[1])};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma16816<__half>(o[nt][4 * wi + j], a, pb0[u][nt], pb1[u][nt]);
        }
      }
    }
  }

  // ---- State exchange of the stream kernel.  A fragment is the float4 (head A dim e, head B dim
  // e, head A dim e + 1, head B dim e + 1) of one lane: kFrags of them per lane cover max(G, 4)
  // heads.
  static constexpr int kHeads = G < 4 ? 4 : G;
  static constexpr int kFrags = kTwice ? KT / 2 : NT * KT;
  // Heads (A; B is the next) and dimension e of fragment f of a lane.
  static __device__ __forceinline__ int frag_head(int f, int lane) {
    const int t = lane & 3;
    return kTwice ? 2 * (t & 1) : f / KT * 8 + 2 * t;
  }
  static __device__ __forceinline__ int frag_dim(int f, int lane) {
    const int mi = kTwice ? f + ((lane & 2) ? KT / 2 : 0) : f % KT;
    return (lane >> 2) * (D / 8) + 2 * mi;
  }
  // Sums l over the lanes of a column, and writes this warp's maxima: m [kHeads][NWARP].
  template <int NWARP>
  __device__ __forceinline__ void put_max(float* m, int warp) {
    const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if (lane < (kTwice ? 2 : 4)) {
        m[(nt * 8 + 2 * t) * NWARP + warp] = mA[nt];
        m[(nt * 8 + 2 * t + 1) * NWARP + warp] = mB[nt];
      }
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        lA[nt] += __shfl_xor_sync(0xffffffffu, lA[nt], off);
        lB[nt] += __shfl_xor_sync(0xffffffffu, lB[nt], off);
        if constexpr (!kTwice) {
          lrA[nt] += __shfl_xor_sync(0xffffffffu, lrA[nt], off);
          lrB[nt] += __shfl_xor_sync(0xffffffffu, lrB[nt], off);
        }
      }
    }
  }
  // Largest of a head's NWARP maxima.
  template <int NWARP>
  static __device__ __forceinline__ float head_max(const float* m, int head) {
    float M = -INFINITY;
#pragma unroll
    for (int q = 0; q < NWARP / 4; ++q) {
      const float4 x = reinterpret_cast<const float4*>(m + head * NWARP)[q];
      M = fmaxf(M, fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)));
    }
    return M;
  }
  // This warp's state relative to the common maxima: frags [kFrags][32], l and lr [kHeads][NWARP].
  template <int NWARP>
  __device__ __forceinline__ void put_state(float4* frags, const float* m, float* l, float* lr, int warp) {
    const int lane = threadIdx.x & 31, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int hA = kTwice ? 2 * (t & 1) : nt * 8 + 2 * t;
      const float MA = head_max<NWARP>(m, hA), MB = head_max<NWARP>(m, hA + 1);
      const float fA = ex2(mA[nt] - MA), fB = ex2(mB[nt] - MB);
      if constexpr (kTwice) {
#pragma unroll
        for (int f = 0; f < kFrags; ++f) {
          float y[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float give = t < 2 ? o[0][f + kFrags][i] : o[0][f][i];
            const float keep = t < 2 ? o[0][f][i] : o[0][f + kFrags][i];
            y[i] = (keep + __shfl_xor_sync(0xffffffffu, give, 2)) * ((i & 1) ? fB : fA);
          }
          frags[f * 32 + lane] = make_float4(y[0], y[1], y[2], y[3]);
        }
      } else {
#pragma unroll
        for (int mi = 0; mi < KT; ++mi)
          frags[(nt * KT + mi) * 32 + lane] = make_float4(o[nt][mi][0] * fA, o[nt][mi][1] * fB,
                                                          o[nt][mi][2] * fA, o[nt][mi][3] * fB);
      }
      if (lane < (kTwice ? 2 : 4)) {
        l[hA * NWARP + warp] = lA[nt] * fA;
        l[(hA + 1) * NWARP + warp] = lB[nt] * fB;
        lr[hA * NWARP + warp] = (kTwice ? lA[nt] : lrA[nt]) * fA;
        lr[(hA + 1) * NWARP + warp] = (kTwice ? lB[nt] : lrB[nt]) * fB;
      }
    }
  }
  template <int NWARP>
  static __device__ __forceinline__ float head_sum(const float* x, int head) {
    float y = 0.f;
#pragma unroll
    for (int q = 0; q < NWARP / 4; ++q) {
      const float4 z = reinterpret_cast<const float4*>(x + head * NWARP)[q];
      y += (z.x + z.y) + (z.z + z.w);
    }
    return y;
  }
  // out[.., e], out[.., e + 1] of a fragment's heads: its values times the heads' 1 / lr.
  static __device__ __forceinline__ void put_out(T* out, int f, int lane, const float4& a, float invA, float invB) {
    const int h = frag_head(f, lane), e = frag_dim(f, lane);
    if (h < G) *reinterpret_cast<uint32_t*>(out + h * D + e) = pack2<T>(a.x * invA, a.z * invA);
    if (h + 1 < G) *reinterpret_cast<uint32_t*>(out + (h + 1) * D + e) = pack2<T>(a.y * invB, a.w * invB);
  }

  // ---- State of the one-CTA-per-partial kernels.
  // Sums over the lanes that share a column; adds the residual columns to theirs.
  __device__ __forceinline__ void finish() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int off = 4; off < 32; off <<= 1) {
        lA[nt] += __shfl_xor_sync(0xffffffffu, lA[nt], off);
        lB[nt] += __shfl_xor_sync(0xffffffffu, lB[nt], off);
        if constexpr (!kTwice) {
          lrA[nt] += __shfl_xor_sync(0xffffffffu, lrA[nt], off);
          lrB[nt] += __shfl_xor_sync(0xffffffffu, lrB[nt], off);
        }
      }
      if constexpr (kTwice) {
        lrA[nt] = lA[nt];
        lrB[nt] = lB[nt];
#pragma unroll
        for (int mi = 0; mi < KT; ++mi)
#pragma unroll
          for (int i = 0; i < 4; ++i) o[nt][mi][i] += __shfl_xor_sync(0xffffffffu, o[nt][mi][i], 2);
      }
    }
  }

  // This warp's state to acc [G][D], m, l and lr [G].
  __device__ __forceinline__ void store(float* acc, float* m, float* l, float* lr) const {
    const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int hA = nt * 8 + 2 * t;
      if (hA < G) {
        float* a = acc + hA * D + g * (D / 8);
#pragma unroll
        for (int mi = 0; mi < KT; ++mi) {
          *reinterpret_cast<float2*>(a + 2 * mi) = make_float2(o[nt][mi][0], o[nt][mi][2]);
          if constexpr (G > 1)
            *reinterpret_cast<float2*>(a + D + 2 * mi) = make_float2(o[nt][mi][1], o[nt][mi][3]);
        }
        if (g == 0) {
          m[hA] = mA[nt];
          l[hA] = lA[nt];
          lr[hA] = lrA[nt];
          if constexpr (G > 1) {
            m[hA + 1] = mB[nt];
            l[hA + 1] = lB[nt];
            lr[hA + 1] = lrB[nt];
          }
        }
      }
    }
  }
};

// ---------------------------------------------------------------------------------------------
// The stream kernel.  A persistent grid of kCtas CTAs per SM; the 128-token tiles of all
// (sequence, KV head) pairs, in that order, are cut into one equal run per CTA, whatever the
// lengths of the sequences; a pair counts kPairUnits tiles more than it has, for the start and
// the end of its piece.  The quads of warps take the tiles of the run in turn, 32 tokens a warp.
// Every warp has a TMA ring of its own and refills a slot as soon as it has read it, across pair
// boundaries: no warp waits for another within a piece, and HBM does not idle while the states of
// a piece are merged.  At the end of a piece the warps' states are merged; a pair that lies in one
// CTA is written at once, else the CTA publishes a record and the last one to arrive at the pair's
// counter combines them, in order.  No CTA waits for another.
//
// What bounds it: HBM for long sequences (64 sequences of 8K tokens, 604 MB, G = 4: 98.6 us, 6.13 TB/s
// of the 6.8 TB/s that a copy reaches; 128K tokens, G = 8: 31.9 us for 151 MB).  The loads alone
// take 90 us there and the arithmetic alone 55 us (238 instructions per block and warp, 104 of
// them on the half-rate ALU pipe), so a slot must not be held for longer than the loads of the
// others take: a warp is done with its 32 tokens in about 2100 cycles; held for 3000, the loads alone
// would take 115 us.  Rings shared by four warps and refilled by the last of them to finish ran at
// 118 us, one CTA per partial (8192 short CTAs) at 212 us.  Short inputs are bound by latencies: one
// 32K-token sequence (G = 4) takes 13.2 us for 38 MB, of which the first loads 2 us, the merge and the
// arrival 2 us and the combine of about 38 records (80 KB) 3 us.
template <int D, int G>
struct Kv4Stream {
  static constexpr int kTile = kStreamTile;
  static constexpr int kWarps = stream_warps(G);
  static constexpr int kCtas = stream_ctas(G);
  static constexpr int kQuads = kWarps / 4;
  static constexpr int kSub = 2;                  // blocks of 16 tokens per warp
  static constexpr int kThreads = kWarps * 32;
  static constexpr int kHeads = G < 4 ? 4 : G;    // of a record (padded)
  static constexpr int kItems = kHeads * D / 4;   // fragments of a state or record
  static constexpr int kRecord = kHeads * (D + 4);  // floats: the fragments, then (m, l, l~, 0) per head
  // The combine: thread (q, l) takes the fragments l, l + kLanes, .. (kPer of them) of every kSplit-th
  // record from q on, sixteen loads at a time.  (G = 16, 21 records: 28 loads per thread, 1.4 us less
  // than with one thread per fragment in two passes.  A load issued as soon as its register is
  // free, instead of sixteen together, was slower: 128K tokens of G = 8 by 3.4 us.)
  static constexpr int kLanes = kItems < (kThreads & -kThreads) ? kItems : (kThreads & -kThreads);
  static constexpr int kPer = kItems / kLanes;
  static constexpr int kSplit = kPer > 1 ? kThreads / kLanes : kThreads / kItems >= 2 ? 2 : 1;
  static constexpr int kDeep = 16 / kPer;
  static constexpr uint32_t kRowsBytes = kSub * 16 * ring_row_bytes(kPathMmaKv4, D);  // K (or V) of a slot
  static constexpr uint32_t kSlotBytes = 2 * kRowsBytes;
  // States of the warps: fragments [kWarps][kItems], m, l, lr [kHeads][kWarps].
  static constexpr uint32_t kStateBytes = kWarps * kHeads * (D + 3) * 4;
  static constexpr uint32_t kMetaBytes = 128 + 1024;  // alignment slack; barriers, cursors and words
  static constexpr int kFit = (int)((228 * 1024 / kCtas - 1024 - kStateBytes - kMetaBytes) / kSlotBytes / kWarps);
  static constexpr int kSlots = kFit < 4 ? kFit : 4;  // per warp
  static constexpr uint32_t kRing = kWarps * kSlots * kSlotBytes;
  static constexpr uint32_t kSmemBytes = kRing + kStateBytes + kMetaBytes;
  // The combine keeps its partial sums and the coefficients [kHeads][records] where the states were.
  static_assert((kWarps - kSplit) * D >= kMaxStreamCtas, "coefficients of the longest pair");
  static_assert(kSlots >= 2 && kWarps * kSlots * 8 + 16 <= 1024, "ring");
  static_assert(kTile == 4 * 16 * kSub && kStreamSlotTokens == 16 * kSub, "a quad covers a tile");
  static_assert(kWarps % 4 == 0 && kStateBytes % 16 == 0, "float4 rows");
};

// Merge of (max, sum, sum) triples with finite maxima.
__device__ __forceinline__ void stream_merge(float& M, float& l, float& lr, float m2, float l2, float lr2) {
  if (m2 > M) {
    const float c = ex2(M - m2);
    l = fmaf(l, c, l2);
    lr = fmaf(lr, c, lr2);
    M = m2;
  } else {
    const float c = ex2(m2 - M);
    l = fmaf(l2, c, l);
    lr = fmaf(lr2, c, lr);
  }
}

// What out is multiplied by for a sum of weights: 0 where no token has any (none there, or all scores
// -inf), so that out is 0; a NaN stays.
__device__ __forceinline__ float stream_inverse(float l) { return l != 0.f ? 1.f / l : 0.f; }

// First unit of CTA c's run: run_len or run_len + 1 of them each.
__device__ __forceinline__ int stream_begin(const Params& p, int c) {
  return c * p.run_len + min(c, p.run_extra);
}
// The CTA whose run holds unit i.
__device__ __forceinline__ int stream_cta(const Params& p, int i) {
  const int cut = p.run_extra * (p.run_len + 1);
  return i < cut ? i / (p.run_len + 1) : p.run_extra + (i - cut) / p.run_len;
}

// A (sequence, KV head) pair on the way through a run: kPairUnits units, then one per tile.
struct StreamPair {
  int b, kvh, units, len;  // its units (one tile, without tokens, for an empty sequence) and tokens
  int at;                  // its first unit in the order of all
  __device__ __forceinline__ void load(const Params& p) {
    len = p.cu[b + 1] - p.cu[b];
    units = (p.unit_base[b + 1] - p.unit_base[b]) / p.Hkv;
  }
  __device__ __forceinline__ void set(const Params& p, int unit) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.unit_base[mid] <= unit) lo = mid; else hi = mid;
    }
    b = lo;
    load(p);
    kvh = (unit - p.unit_base[b]) / units;
    at = p.unit_base[b] + kvh * units;
  }
  __device__ __forceinline__ void next(const Params& p) {
    at += units;
    if (++kvh == p.Hkv) {
      kvh = 0;
      if (++b < p.B) load(p);
    }
  }
  __device__ __forceinline__ int first_tile(int unit) const { return max(0, unit - at - kPairUnits); }
};

// What a warp loads next: its 32 tokens of tiles i, i + kQuads, .. of pair sp, `left` more of
// them, then those of the following pairs; `row` is the next load's TMA row (its first token where
// the cache is paged).  Every lane holds the same values, so that they can live in uniform registers
// (contiguous caches; the paged kernels keep the cursor in 40 bytes of local memory, because stream_load
// indexes page[] at run time).
template <bool PAGED>
struct StreamCursor {
  StreamPair sp;
  int i, left, row;
  int page[2];  // paged caches: TMA rows of the next load's 16-token halves, read one load ahead
  // On by n tiles that hold tokens; i >= end when the run has fewer.
  __device__ __forceinline__ void seek(const Params& p, int n, int end) {
    while (i < end) {
      i = max(i, sp.at + kPairUnits);
      const int left = sp.len > 0 ? sp.at + sp.units - i : 0;
      if (n < left) {
        i += n;
        return;
      }
      n -= max(left, 0);
      i = sp.at + sp.units;
      sp.next(p);
    }
  }
  // The batch that starts at or after i (left = 0: the run is done).
  __device__ __forceinline__ void batch(const Params& p, int quads, int first_token, int end) {
    for (left = 0; i < end; seek(p, quads, end)) {
      // Tiles of the pair, within the run, in which this warp has tokens.
      const int tile = i - sp.at - kPairUnits;
      const int tiles = min((sp.len - first_token + kStreamTile - 1) / kStreamTile, end - sp.at - kPairUnits);
      if (sp.len > first_token && tile < tiles) {
        const int token = tile * kStreamTile + first_token;
        row = PAGED ? token : p.blk[sp.b] + token / kBlockTokens;
        left = (tiles - tile - 1) / quads + 1;
        return;
      }
    }
  }
  // Page-table entries of the next load; pages past the end of the sequence: its last one.
  __device__ __forceinline__ void read_pages(const Params& p) {
    if (!PAGED || left == 0) return;
    const int32_t* bt = p.block_table + (int64_t)sp.b * p.bt_stride;
    const int last_pg = (sp.len - 1) >> p.page_shift;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int a = row + k * kBlockTokens, pg = min(a >> p.page_shift, last_pg);
      // An index that no pool has goes to a row outside every pool (TMA reads zeros there).
      const int entry = __ldg(bt + pg);
      const bool possible = (uint32_t)entry <= (0x7fffffffu >> p.page_shift);
      page[k] = possible ? ((entry << p.page_shift) + (a & ((1 << p.page_shift) - 1))) >> kBlockShift : -kBlockTokens;
    }
  }
  // Past one load.
  __device__ __forceinline__ void step(const Params& p, int quads, int first_token, int end) {
    row += quads * (PAGED ? kStreamTile : kStreamTile / kBlockTokens);
    i += quads;
    if (--left == 0) {
      i -= quads;
      seek(p, quads, end);
      batch(p, quads, first_token, end);
    }
    read_pages(p);
  }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

// K and V of one slot (32 tokens of a KV head) to dst.
template <int D, int G, bool PAGED>
__device__ __forceinline__ void stream_load(const Params& p, const StreamCursor<PAGED>& cur, uint32_t dst, uint32_t bar,
                                            uint64_t policy) {
  using S = Kv4Stream<D, G>;
  const int kvh = cur.sp.kvh;
  mbar_arrive_expect_tx(bar, S::kSlotBytes);
  if constexpr (!PAGED) {
    tma_load_3d(dst, &p.tm_k, 0, kvh, cur.row, bar, policy);
    tma_load_3d(dst + S::kRowsBytes, &p.tm_v, 0, kvh, cur.row, bar, policy);
  } else {
    // Pages of 16 tokens: a box for each half of the slot; larger pages hold all of it.
    for (int k = 0; k * p.box_rows < kStreamSlotTokens; ++k) {
      const uint32_t to = dst + k * kBlockTokens * ring_row_bytes(kPathMmaKv4, D);
      tma_load_3d(to, &p.tm_k, 0, kvh, cur.page[k], bar, policy);
      tma_load_3d(to + S::kRowsBytes, &p.tm_v, 0, kvh, cur.page[k], bar, policy);
    }
  }
}

template <typename T, int D, int G, bool PAGED>
__global__ void __launch_bounds__((Kv4Stream<D, G>::kThreads), (Kv4Stream<D, G>::kCtas))
    fd_kv4_stream_kernel(const __grid_constant__ Params p) {
  using S = Kv4Stream<D, G>;
  using W = Kv4Warp<T, D, G>;
  constexpr int kTile = S::kTile, NSLOT = S::kSlots, NW = S::kWarps, H = S::kHeads;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((128u - (smem_addr(smem_raw) & 127u)) & 127u);
  float4* st_frag = reinterpret_cast<float4*>(smem + S::kRing);  // [NW][kItems]
  float* st_m = reinterpret_cast<float*>(st_frag + NW * S::kItems);           // [H][NW], then l, lr
  float* st_l = st_m + H * NW;
  float* st_lr = st_l + H * NW;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::kRing + S::kStateBytes);  // [NW][NSLOT]
  volatile int* words = reinterpret_cast<volatile int*>(bars + NW * NSLOT);        // abort, role

  // The warp index through a shuffle: the compiler then knows that it is uniform.
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  const int quad = warp >> 2, first_token = (warp & 3) * 16 * S::kSub;
  pdl_launch_dependents();
  const int c = blockIdx.x, i0 = stream_begin(p, c), i1 = stream_begin(p, c + 1);
  const uint32_t bar = smem_addr(bars + warp * NSLOT), ring = smem_addr(smem + warp * NSLOT * S::kSlotBytes);
  StreamPair sp;
  sp.set(p, i0);
  const uint64_t policy = l2_evict_first_policy();
  int loads = 0;
  if (lane == 0) {
    for (int s = 0; s < NSLOT; ++s) mbar_init(bar + 8 * s, 1);
    fence_mbar_init();
    if (tid == 0) words[0] = 0;
  }
  // The warp's loads, one slot after the other.
  StreamCursor<PAGED> cur;
  cur.sp = sp;
  cur.i = i0;
  cur.seek(p, quad, i1);
  cur.batch(p, S::kQuads, first_token, i1);
  // The first slot into L2 while the previous kernel drains (see fd_split_kernel).
  if (cur.left > 0 && lane == 0) {
    prefetch_tensormap(&p.tm_k);
    prefetch_tensormap(&p.tm_v);
    if (!PAGED) {
      tma_prefetch_l2_3d(&p.tm_k, 0, cur.sp.kvh, cur.row);
      tma_prefetch_l2_3d(&p.tm_v, 0, cur.sp.kvh, cur.row);
    }
  }
  if (p.test_hook == kHookSkipTile && c == 0 && warp == 4) cur.left = 0;  // test hook: loads nothing
  auto load_next = [&](int slot) {
    if (cur.left == 0) return;
    if (elect_one())
      stream_load<D, G, PAGED>(p, cur, ring + slot * S::kSlotBytes, bar + 8 * slot, policy);
    __syncwarp();
    cur.step(p, S::kQuads, first_token, i1);
    ++loads;
  };
  __syncwarp();
  pdl_wait();  // q, K, V, the workspace and out may come from earlier kernels
  cur.read_pages(p);
  // q ahead of K and V: behind them it would wait for the whole ring (3 us when all CTAs start).
  W w;
  w.fetch_q(p, sp.b, sp.kvh);
#pragma unroll 1
  for (int s = 0; s < NSLOT; ++s) load_next(s);
  __syncthreads();

  bool gave_up = false;
  int turn = quad;     // tiles of the run until the quad's next one
  int slot = 0;        // the warp's next slot, and the parity of its barrier
  uint32_t parity = 0;
  // Pairs that other CTAs share: the arrival's answer, read at the end of the run.
  uint32_t arrived0 = 0, arrived1 = 0;  // thread 0's
  StreamPair shared0 = sp, shared1 = sp;
  int n_shared = 0;
#pragma unroll 1
  for (int i = i0; i < i1;) {
    const int end = min(i1, sp.at + sp.units);
    const int ta = sp.first_tile(i), nt = sp.first_tile(end) - ta;
    i = end;
    if (nt <= 0) break;  // the run ends before the pair's first tile
    w.start(p);
    if (sp.len > 0) {
      int ntok = sp.len - (ta + turn) * kTile - first_token;
#pragma unroll 1
      for (; turn < nt; turn += S::kQuads, ntok -= S::kQuads * kTile) {
        if (ntok <= 0 || gave_up) continue;
        if (!__all_sync(0xffffffffu, mbar_wait(bar + 8 * slot, parity))) {
          atomicOr(p.status, kStatusTimeout);
          words[0] = 1;
          gave_up = true;
          continue;
        }
        const uint8_t* kblk = smem + (warp * NSLOT + slot) * S::kSlotBytes;
        w.template blocks<S::kSub>(kblk, kblk + S::kRowsBytes, ntok);
        __syncwarp();  // every lane has read the slot
        load_next(slot);
        if (++slot == NSLOT) {
          slot = 0;
          parity ^= 1;
        }
      }
      turn -= nt;
    }
    const StreamPair done = sp;
    sp.next(p);
    // The next piece's q, on its way while the states are merged.
    if (i < i1) w.fetch_q(p, sp.b, sp.kvh);
    // Merge the warps' states: common maxima first, then plain sums.
    w.template put_max<NW>(st_m, warp);
    __syncthreads();
    w.template put_state<NW>(st_frag + warp * S::kItems, st_m, st_l, st_lr, warp);
    __syncthreads();
    const bool aborted = words[0] != 0;  // a CTA that gave up contributes empty partials
    const bool whole = ta == 0 && nt == done.units - kPairUnits;
    T* out = reinterpret_cast<T*>(p.out) + ((int64_t)done.b * p.Hq + done.kvh * G) * D;
    float* lse = p.lse == nullptr ? nullptr : p.lse + (int64_t)done.b * p.Hq + done.kvh * G;
    // Record 0 of a CTA: of a piece whose pair begins no later than its run; record 1: of its last.
    float* rec = p.part + ((int64_t)c * 2 + (i0 >= done.at ? 0 : 1)) * S::kRecord;
    for (int v = tid; v < S::kItems; v += S::kThreads) {
      float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
      if (!aborted) {
#pragma unroll
        for (int q = 0; q < NW; ++q) {
          const float4 x = st_frag[q * S::kItems + v];
          a.x += x.x; a.y += x.y; a.z += x.z; a.w += x.w;
        }
      }
      if (whole) {
        const int h = W::frag_head(v >> 5, lane);
        const float lA = aborted ? 0.f : W::template head_sum<NW>(st_lr, h);
        const float lB = aborted ? 0.f : W::template head_sum<NW>(st_lr, h + 1);
        W::put_out(out, v >> 5, lane, a, stream_inverse(lA), stream_inverse(lB));
      } else {
        __stcg(reinterpret_cast<float4*>(rec) + v, a);
      }
    }
    if (tid < H) {
      const float M = aborted ? -INFINITY : W::template head_max<NW>(st_m, tid);
      const float l = aborted ? 0.f : W::template head_sum<NW>(st_l, tid);
      if (whole) {
        if (lse != nullptr && tid < G) lse[tid] = l != 0.f ? (M + log2f(l)) * kLn2 : -INFINITY;
      } else {
        const float lr = aborted ? 0.f : W::template head_sum<NW>(st_lr, tid);
        __stcg(reinterpret_cast<float4*>(rec + H * D) + tid, make_float4(M, l, lr, 0.f));
      }
    }
    __syncthreads();  // the next piece overwrites the states
    if (!whole) {
      // Arrival, as in finish_cta: the barrier orders the CTA's stores before thread 0's release.
      // Whether this CTA was the last of the pair is asked at the end of its run.
      if (tid == 0) {
        const uint32_t old = atom_add_acq_rel_gpu(p.counters + (int64_t)done.b * p.Hkv + done.kvh, 1u);
        if (n_shared == 0) arrived0 = old; else arrived1 = old;
      }
      if (n_shared == 0) shared0 = done; else shared1 = done;
      ++n_shared;
    }
  }

  // The pairs that this CTA shares with others and was the last to arrive at: combine their
  // records, in CTA order.  Only a pair's first CTA can have begun before it.
#pragma unroll 1
  for (int k = 0; k < n_shared; ++k) {
    const StreamPair pr = k == 0 ? shared0 : shared1;
    const int c_first = stream_cta(p, pr.at + kPairUnits), nrec = stream_cta(p, pr.at + pr.units - 1) - c_first + 1;
    if (tid == 0) {
      const uint32_t old = k == 0 ? arrived0 : arrived1;
      if (old >= (uint32_t)nrec) atomicOr(p.status, kStatusCounter);
      const bool last = old == (uint32_t)(nrec - 1);
      if (last) p.counters[(int64_t)pr.b * p.Hkv + pr.kvh] = 0u;  // every CTA of the pair has arrived
      words[1] = last;
    }
    __syncthreads();
    const bool last = words[1] != 0;
    __syncthreads();
    if (!last) continue;
    T* out = reinterpret_cast<T*>(p.out) + ((int64_t)pr.b * p.Hq + pr.kvh * G) * D;
    float* lse = p.lse == nullptr ? nullptr : p.lse + (int64_t)pr.b * p.Hq + pr.kvh * G;
    float4* sums = st_frag;                                                    // [kSplit][kItems]
    float* coef = reinterpret_cast<float*>(st_frag + S::kSplit * S::kItems);   // [H][nrec]
    const float* rec1 = p.part + (int64_t)c_first * 2 * S::kRecord;
    const float* rec0 = rec1 + (stream_begin(p, c_first) >= pr.at ? 0 : S::kRecord);
    auto record = [&](int r) { return r == 0 ? rec0 : rec1 + (int64_t)r * 2 * S::kRecord; };
    const int q = tid / S::kLanes, l0 = tid % S::kLanes;
    // Maxima and sums of this warp's heads, then the first fragments, are on their way together.
    constexpr int kMine = (H + NW - 1) / NW;
    auto sums_of = [&](int g, int r) {
      float4 y = __ldcg(reinterpret_cast<const float4*>(record(r) + H * D) + g);
      y.x = fmaxf(y.x, -FLT_MAX);  // -inf: a CTA that gave up
      return y;
    };
    float4 ml[kMine];
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      ml[j] = make_float4(-FLT_MAX, 0.f, 0.f, 0.f);
      if (warp + j * NW < H && lane < nrec) ml[j] = sums_of(warp + j * NW, lane);
    }
    float4 x[S::kDeep][S::kPer];
    auto fetch = [&](int u, int r) {
      if (r >= nrec) return;
      const float4* src = reinterpret_cast<const float4*>(record(r)) + l0;
#pragma unroll
      for (int j = 0; j < S::kPer; ++j) x[u][j] = __ldcg(src + j * S::kLanes);
    };
    const int r_first = q < S::kSplit ? q : nrec;
#pragma unroll
    for (int u = 0; u < S::kDeep; ++u) fetch(u, r_first + u * S::kSplit);
#pragma unroll
    for (int j = 0; j < kMine; ++j) {
      const int g = warp + j * NW;
      if (g >= H) break;
      float M = ml[j].x, l = ml[j].y, lr = ml[j].z;
      if (lane < nrec) coef[g * nrec + lane] = M;
      for (int r = lane + 32; r < nrec; r += 32) {
        const float4 y = sums_of(g, r);
        coef[g * nrec + r] = y.x;
        stream_merge(M, l, lr, y.x, y.y, y.z);
      }
      const float own = M;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, off));
      const float c = ex2(own - M);
      l *= c;
      lr *= c;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) {
        l += __shfl_xor_sync(0xffffffffu, l, off);
        lr += __shfl_xor_sync(0xffffffffu, lr, off);
      }
      for (int r = lane; r < nrec; r += 32) coef[g * nrec + r] = ex2(coef[g * nrec + r] - M);
      if (lane == 0) {
        st_lr[g] = lr;
        if (lse != nullptr && g < G) lse[g] = l != 0.f ? (M + log2f(l)) * kLn2 : -INFINITY;
      }
    }
    __syncthreads();
    float4 a[S::kPer];
    int head[S::kPer];
#pragma unroll
    for (int j = 0; j < S::kPer; ++j) {
      a[j] = make_float4(0.f, 0.f, 0.f, 0.f);
      head[j] = W::frag_head((l0 + j * S::kLanes) >> 5, lane);
    }
#pragma unroll 1
    for (int r0 = r_first; r0 < nrec; r0 += S::kDeep * S::kSplit) {
      if (r0 != r_first)
#pragma unroll
        for (int u = 0; u < S::kDeep; ++u) fetch(u, r0 + u * S::kSplit);
#pragma unroll
      for (int u = 0; u < S::kDeep; ++u) {
        const int r = r0 + u * S::kSplit;
        if (r < nrec) {
#pragma unroll
          for (int j = 0; j < S::kPer; ++j) {
            const float fA = coef[head[j] * nrec + r], fB = coef[(head[j] + 1) * nrec + r];
            a[j].x = fmaf(x[u][j].x, fA, a[j].x);
            a[j].y = fmaf(x[u][j].y, fB, a[j].y);
            a[j].z = fmaf(x[u][j].z, fA, a[j].z);
            a[j].w = fmaf(x[u][j].w, fB, a[j].w);
          }
        }
      }
    }
    if constexpr (S::kSplit == 1) {
#pragma unroll
      for (int j = 0; j < S::kPer; ++j)
        W::put_out(out, (l0 + j * S::kLanes) >> 5, lane, a[j], stream_inverse(st_lr[head[j]]),
                   stream_inverse(st_lr[head[j] + 1]));
    } else {
      if (q < S::kSplit)
#pragma unroll
        for (int j = 0; j < S::kPer; ++j) sums[q * S::kItems + j * S::kLanes + l0] = a[j];
      __syncthreads();
      for (int v = tid; v < S::kItems; v += S::kThreads) {
        float4 y = sums[v];
#pragma unroll
        for (int k = 1; k < S::kSplit; ++k) {
          const float4 z = sums[k * S::kItems + v];
          y.x += z.x; y.y += z.y; y.z += z.z; y.w += z.w;
        }
        const int h = W::frag_head(v >> 5, lane);
        W::put_out(out, v >> 5, lane, y, stream_inverse(st_lr[h]), stream_inverse(st_lr[h + 1]));
      }
    }
    __syncthreads();  // the next pair overwrites the sums
  }
  // A warp that gave up leaves loads behind: they must land before shared memory is released.
  if (gave_up && lane == 0)
    for (int s = 0; s < NSLOT; ++s) {
      const int n = (loads - s + NSLOT - 1) / NSLOT;  // loads of slot s
      if (n > 0) mbar_wait(bar + 8 * s, (n - 1) & 1);
    }
}

}  // namespace dev
}  // namespace fd
