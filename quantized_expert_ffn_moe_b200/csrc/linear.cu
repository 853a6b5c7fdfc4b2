// Products of few token rows with a packed 4-bit matrix: a plain linear layer
// and the gate/up half of a gated feed-forward block.
//
//   z[t][n] = rs_n * sum_b s_{n,b} * sum_{k in block b} q_{n,k} x[t][k]
//   linear: y[t][n] = z[t][n] (+ bias[n]);   gated: h[t][i] = silu(z[t][2i]) * z[t][2i+1]
//
// (q the code's level, s the block's scale, rs the row scale of the fp8
// format.)  Bound by the packed bytes, n * k / 2 plus the scales.
//
// A warp multiplies 16 rows at a time with the warp-level tensor instruction
// m16n8k16 (fp16 operands, fp32 accumulation), rows as M and up to 8 tokens as
// N, one 32-element block per two instructions, so that a block's sum comes
// out by itself and its scale enters fp32 with one multiply-add per row and
// token.  The instruction issues every 2 cycles per SM (measured); the HBM
// rate brings 16 rows x 16 codes every 5.5 cycles, so up to two groups of 8
// tokens run below the memory bound and dequantising is what must be cheap:
// eight codes become exact fp16 integers with four masks, one shift and four
// half2 operations.  (Fed as they are, as fp16 subnormals, with the offset
// taken off through the accumulator, they cost half of that, but the sums
// then carry the offset's magnitude: 4 to 8 times the rounding error.)
// The k order inside a block is free as long as both operands share it: lane
// t of a row's quad takes the block's t-th 32-bit word, as stored.
//
// Activations become fp16 after the power of two that brings the row's largest
// magnitude into [2^13, 2^14): exact for every element within 2^-27 of that
// largest one, off by at most 2^-38 of it below (fp32 sums lose more).  A row
// with an infinity or a NaN gives NaN in all its outputs.
//
// Each warp streams its own stages of 16 rows x 128 or 256 columns through a
// private ring of asynchronous copies (no block-wide barrier in the stream);
// the warps of a group split the columns of a row tile, so that even 2048 x
// 2048 spreads over 128 SMs, and join their fp32 sums through shared memory in
// a fixed order: the same inputs give the same bits.
#include "dense_internal.cuh"

namespace moe {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr size_t kMaxSmem = 232448;

// scale formats: fp16 per 32, fp16 per 128, E4M3 per 32 under a row scale; the
// fp16 ones with integer or half-integer levels
enum { F_H32 = 0, F_H128 = 1, F_E32 = 2, F_H32_HALF = 3, F_H128_HALF = 4 };
template <int FMT>
struct Format {
  static constexpr bool HALF = FMT == F_H32_HALF || FMT == F_H128_HALF;
  static constexpr bool G128 = FMT == F_H128 || FMT == F_H128_HALF;
  static constexpr int SB = FMT == F_E32 ? 1 : 2;            // bytes of a scale
};
// A stage: 16 rows x CB blocks of 32 columns, codes then scales (up to CB fp16
// a row), in a ring of ST slots per warp.  8 blocks halve the per-stage work;
// 4 leave room for more activations.
template <int CB>
struct Stage {
  static constexpr int ROW = CB * 16;
  static constexpr int CODES = 16 * ROW;
  static constexpr int BYTES = CODES + 32 * CB;
  static constexpr int ST = CB == 8 ? 3 : 4;
  static constexpr int RING = kWarps * ST * BYTES;
};

struct LinearArgs {
  const uint8_t* codes;
  const void* scales;
  const float* row_scales;
  const float* bias;
  const void* x;
  void* y;
  int N, K, T;          // matrix rows, columns, token rows
  int nb;               // 32-element blocks of a row
  int spr;              // scales of a row
  int chunks;           // stages of a row
  int KG, groups;       // warps splitting a row tile's columns; row tiles in flight per CTA
  int ny, tt;           // token slices, tokens of a slice
  int x_type, y_type, gated;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int B>
__device__ __forceinline__ void cp_async_small(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(B) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// d = a b + c; c = 0 where the sum starts (zeros that stay in registers)
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1, float c0,
                                         float c1, float c2, float c3) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Eight codes as exact fp16 pairs (e_j, e_{j+4}), j = 0..3.  Integer levels:
// c - 8; half-integer levels: 2 c - 15, twice the level (halved at the end).
// A 16-bit lane 0x6400 | m is 1024 + m.
template <bool HALF>
__device__ __forceinline__ void levels(uint32_t w, uint32_t (&q)[4]) {
  if (!HALF) {
    __half2 h[4];
    decode_q4x8(w, h);
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = h2_as_u32(h[j]);
  } else {
    const uint32_t MAGIC = 0x64006400u;
    const __half2 sub = u32_as_h2(0x640F640Fu);                                    // 1039 = 1024 + 15
    const __half2 mul = u32_as_h2(0x30003000u), add = u32_as_h2(0xD878D878u);      // 1/8, -143 = -(128 + 15)
    q[0] = h2_as_u32(__hsub2(u32_as_h2(lop_and_or(w << 1, 0x001E001Eu, MAGIC)), sub));
    q[1] = h2_as_u32(__hfma2(u32_as_h2(lop_and_or(w, 0x00F000F0u, MAGIC)), mul, add));
    q[2] = h2_as_u32(__hsub2(u32_as_h2(lop_and_or(w >> 7, 0x001E001Eu, MAGIC)), sub));
    q[3] = h2_as_u32(__hfma2(u32_as_h2(lop_and_or(w >> 8, 0x00F000F0u, MAGIC)), mul, add));
  }
}

// Scales of a row's blocks in a stage as floats (one for all with groups of
// 128 and CB = 4, two with CB = 8).
template <int FMT, int CB>
__device__ __forceinline__ void stage_scales(const unsigned char* sc, int row, float (&s)[CB]) {
  if (Format<FMT>::G128) {
    const __half* p = reinterpret_cast<const __half*>(sc) + row * (CB / 4);
    const float a = __half2float(p[0]), b = CB == 8 ? __half2float(p[1]) : a;
#pragma unroll
    for (int i = 0; i < CB; ++i) s[i] = i < 4 ? a : b;
  } else {
    uint32_t w[CB / 2];
    if (FMT == F_E32) {
#pragma unroll
      for (int i = 0; i < CB / 4; ++i) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(sc + row * CB + 4 * i);
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t"
            "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(w[2 * i]), "=r"(w[2 * i + 1]) : "r"(v));
      }
    } else if (CB == 8) {
      const uint4 v = *reinterpret_cast<const uint4*>(sc + row * 16);
      w[0] = v.x; w[1] = v.y; w[CB / 2 - 2] = v.z; w[CB / 2 - 1] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(sc + row * 8);
      w[0] = v.x; w[1] = v.y;
    }
#pragma unroll
    for (int i = 0; i < CB / 2; ++i) {
      const float2 f = __half22float2(u32_as_h2(w[i]));
      s[2 * i] = f.x;
      s[2 * i + 1] = f.y;
    }
  }
}

// Shared memory: ring | x [tt][nb | 1][4] 16-byte words (an odd number of
// blocks, so that two tokens' words fall into different banks) | partial sums [groups
// KG][16][8 NT] floats | inv [8 NT] floats | row maxima [tt][16] u32.
inline size_t linear_smem(int ring, int nb, int tt, int nt) {
  return size_t(ring) + size_t(nb | 1) * tt * 64 + size_t(kWarps) * 16 * 8 * nt * 4 + size_t(nt) * 32 + size_t(tt) * 64;
}

// Eight activations as fp16 pairs (j, j + 4), the order of `levels`.
__device__ __forceinline__ uint4 pack_activations(const uint4& v, bool bf, float mul) {
  const uint32_t q[4] = {v.x, v.y, v.z, v.w};
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf) {
      f[2 * i] = __uint_as_float(q[i] << 16);
      f[2 * i + 1] = __uint_as_float(q[i] & 0xffff0000u);
    } else {
      const float2 h = __half22float2(u32_as_h2(q[i]));
      f[2 * i] = h.x;
      f[2 * i + 1] = h.y;
    }
  }
  uint32_t o[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = h2_as_u32(__floats2half2_rn(f[j] * mul, f[j + 4] * mul));
  return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int NT, int FMT, int CB>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const LinearArgs a) {
  using F = Format<FMT>;
  using S = Stage<CB>;
  extern __shared__ __align__(128) unsigned char lsm[];
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) >> 5, 0), lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int nb = a.nb, tt = a.tt;
  constexpr int TP = 8 * NT;
  unsigned char* sx = lsm + S::RING;
  float* spart = reinterpret_cast<float*>(sx + (nb | 1) * tt * 64);
  float* sinv = spart + kWarps * 16 * TP;
  uint32_t* smax = reinterpret_cast<uint32_t*>(sinv + TP);

  const int xpitch = (nb | 1) * 64;
  const int slice = int(blockIdx.x % unsigned(a.ny)), cta = int(blockIdx.x / unsigned(a.ny));
  const int ctas = int(gridDim.x / unsigned(a.ny));
  const int t0 = slice * tt, nt = min(tt, a.T - t0);     // this CTA's tokens
  const int ntiles = (a.N + 15) >> 4;
  const int grp = warp / a.KG, kw = warp - grp * a.KG;
  // neighbouring tiles go to different CTAs, so that CTAs differ by one tile at most
  const int first = grp * ctas + cta, step = ctas * a.groups;
  const int my_chunks = grp < a.groups ? (a.chunks - kw + a.KG - 1) / a.KG : 0;
  const int my_tiles = grp < a.groups && first < ntiles ? (ntiles - first + step - 1) / step : 0;
  const int total = my_tiles * my_chunks;

  // ------------------------------------------------------ weight stream
  // This lane copies CB / 4 x 2 16-byte pieces of a stage's codes: piece
  // `ch` of the rows r0 + i * RS, swizzled so that the words of eight rows
  // fall into different banks.
  unsigned char* ring = lsm + warp * (S::ST * S::BYTES);
  const uint32_t ring_s = smem_u32(ring);
  constexpr int RS = 32 / CB;                             // rows covered by one warp-wide copy
  const int r0 = lane / CB, ch = lane % CB;
  const int row_bytes = a.K >> 1;
  constexpr int SPC = F::G128 ? CB / 4 : CB;              // scales of a row in a stage
  // scales that cannot be copied asynchronously (rows off the copy's
  // alignment, or one fp16 per stage) pass through registers: loaded with
  // their stage's codes, stored to its slot when the next stage is issued
  constexpr bool kMayCopy = SPC * F::SB >= 4;
  const bool direct = kMayCopy && a.spr % SPC == 0;
  constexpr int PEND = (16 * SPC + 31) / 32;
  uint16_t pend[PEND];
  int pend_slot = -1;
  auto flush_pending = [&]() {
    if (pend_slot < 0) return;
    unsigned char* sc = ring + pend_slot * S::BYTES + S::CODES;
#pragma unroll
    for (int i = 0; i < PEND; ++i) {
      const int e = i * 32 + lane;
      if (e < 16 * SPC) {
        if (F::SB == 2) *reinterpret_cast<uint16_t*>(sc + e * 2) = pend[i];
        else sc[e] = uint8_t(pend[i]);
      }
    }
    pend_slot = -1;
  };
  const uint8_t* src = nullptr;      // this lane's piece of the next stage, row r0 of its tile
  const uint8_t* ssrc = nullptr;     // (direct) the scales of row `lane` of that tile
  int it_tile = first, it_chunk = 0, left = total, slot_i = 0;
  int row_off[CB / 2];               // from row r0 to this lane's other rows; rows past the end: the last one again
  uint32_t dst_off[CB / 2];
#pragma unroll
  for (int i = 0; i < CB / 2; ++i) {
    const int r = r0 + i * RS;
    row_off[i] = i * RS * row_bytes;
    dst_off[i] = r * S::ROW + ((ch ^ (CB == 8 ? r & 7 : (r >> 1) & 3)) << 4);
  }
  auto enter_tile = [&]() {
    it_chunk = kw;
    if (it_tile * 16 + 16 > a.N) {
#pragma unroll
      for (int i = 0; i < CB / 2; ++i) row_off[i] = min(i * RS, a.N - 1 - it_tile * 16 - r0) * row_bytes;
    }
    src = a.codes + size_t(it_tile * 16 + r0) * row_bytes + size_t(kw) * S::ROW + ch * 16;
    ssrc = static_cast<const uint8_t*>(a.scales) +
           (size_t(min(it_tile * 16 + (lane & 15), a.N - 1)) * a.spr + size_t(kw) * SPC) * F::SB;
  };
  if (left > 0) enter_tile();
  auto issue = [&]() {
    if (!direct) flush_pending();
    if (left > 0) {
      const uint32_t dst = ring_s + slot_i * S::BYTES;
      if (it_chunk * CB + ch < nb) {                      // the last stage of a row may be short
#pragma unroll
        for (int i = 0; i < CB / 2; ++i) cp_async16(dst + dst_off[i], src + row_off[i]);
      }
      if (direct) {
        if (lane < 16) {
          constexpr int B = kMayCopy ? SPC * F::SB : 4;
          if (B == 16) cp_async16(dst + S::CODES + lane * 16, ssrc);
          else cp_async_small<B == 16 ? 8 : B>(dst + S::CODES + lane * B, ssrc);
        }
      } else {
#pragma unroll
        for (int i = 0; i < PEND; ++i) {
          const int e = i * 32 + lane, b = it_chunk * SPC + e % SPC;
          pend[i] = 0;
          if (e < 16 * SPC && b < a.spr) {
            const size_t at = size_t(min(it_tile * 16 + e / SPC, a.N - 1)) * a.spr + b;
            pend[i] = F::SB == 2 ? ld_stream2(static_cast<const uint16_t*>(a.scales) + at)
                                 : uint16_t(__ldg(static_cast<const uint8_t*>(a.scales) + at));
          }
        }
        pend_slot = slot_i;
      }
      --left;
      slot_i = slot_i + 1 == S::ST ? 0 : slot_i + 1;
      it_chunk += a.KG;
      src += a.KG * S::ROW;
      ssrc += a.KG * SPC * F::SB;
      if (it_chunk >= a.chunks) {
        it_tile += step;
        if (left > 0) enter_tile();
      }
    }
    cp_async_commit();
  };
  // the weights do not depend on the previous kernel of the stream
#pragma unroll
  for (int s = 0; s < S::ST - 1; ++s) issue();

  pdl_wait();
  pdl_launch_dependents();

  // ------------------------------------------------------ activations
  // A unit is (token, slice of its columns); with fewer tokens than warps a
  // token's columns are split over several warps.  A unit's words are held in
  // registers between the maximum and the conversion when they fit there.
  {
    constexpr int HOLD = 8;
    const int sl = nt >= kWarps ? 1 : kWarps / nt;         // slices of a token
    const int units = nt * sl;
    const int K8 = a.K >> 3;                               // 16-byte words of a token row
    const int per = (K8 + sl - 1) / sl;
    const bool bf = a.x_type == MOE_BF16;
    const uint16_t* xb = static_cast<const uint16_t*>(a.x) + size_t(t0) * a.K;
    const bool held = units <= kWarps && per <= HOLD * 32;
    uint4 hold[HOLD];
    auto word_max = [](uint32_t m, const uint4& v) {
      const uint32_t q = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                  __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
      return __vmaxu2(m, q);
    };
    for (int u = warp; u < units; u += kWarps) {
      const int n = u / sl, p = u % sl, end = min(K8, (p + 1) * per);
      const uint4* src8 = reinterpret_cast<const uint4*>(xb + size_t(n) * a.K);
      uint32_t m = 0;
      for (int w0 = p * per; w0 < end; w0 += HOLD * 32) {
#pragma unroll
        for (int i = 0; i < HOLD; ++i) {
          const int w = w0 + i * 32 + lane;
          hold[i] = w < end ? __ldg(src8 + w) : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < HOLD; ++i) m = word_max(m, hold[i]);
      }
      m = __reduce_max_sync(0xffffffffu, max(m & 0xffffu, m >> 16));
      if (lane == 0) smax[n * 16 + p] = m;
    }
    __syncthreads();
    for (int u = warp; u < units; u += kWarps) {
      const int n = u / sl, p = u % sl, end = min(K8, (p + 1) * per);
      uint32_t m = lane < sl ? smax[n * 16 + lane] : 0u;
      m = __reduce_max_sync(0xffffffffu, m);
      const bool finite = m < (bf ? 0x7f80u : 0x7c00u);
      const float top = bf ? __uint_as_float(m << 16) : __half2float(__ushort_as_half((unsigned short)m));
      int sh = 0;
      if (finite && top > 0.f) {
        int ex;
        frexpf(top, &ex);
        sh = min(max(14 - ex, -120), 120);
      }
      const float mul = ldexpf(1.f, sh);
      if (p == 0 && lane == 0) sinv[n] = finite ? ldexpf(F::HALF ? 0.5f : 1.f, -sh) : __int_as_float(0x7fc00000);
      const uint4* src8 = reinterpret_cast<const uint4*>(xb + size_t(n) * a.K);
      for (int w0 = p * per; w0 < end; w0 += HOLD * 32) {
        if (!held) {
#pragma unroll
          for (int i = 0; i < HOLD; ++i) {
            const int w = w0 + i * 32 + lane;
            if (w < end) hold[i] = __ldg(src8 + w);
          }
        }
#pragma unroll
        for (int i = 0; i < HOLD; ++i) {
          const int w = w0 + i * 32 + lane;
          if (w < end)
            *reinterpret_cast<uint4*>(sx + n * xpitch + w * 16) = pack_activations(hold[i], bf, mul);
        }
      }
    }
    __syncthreads();
  }
  if (total == 0) return;             // whole warps; a group's warps leave together

  // ------------------------------------------------------------ stream
  // this lane's words of the tokens 8 j + g (the last token's where there is
  // none: those columns are never stored)
  const unsigned char* xrow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xrow[j] = sx + min(8 * j + g, nt - 1) * xpitch + t * 16;
  const uint32_t lane_code = uint32_t(g * S::ROW + ((CB == 8 ? g : (g >> 1) & 3) << 4) + t * 4);
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

  int tile = first, chunk = kw, slot = 0;
  bool first_tile = true;
  for (int it = 0; it < total; ++it) {
    __syncwarp();                     // every lane is done with the slot that is filled next
    issue();
    cp_async_wait<S::ST - 1>();
    __syncwarp();
    const unsigned char* st = ring + slot * S::BYTES;
    slot = slot + 1 == S::ST ? 0 : slot + 1;
    float s0[CB], s1[CB];
    stage_scales<FMT, CB>(st + S::CODES, g, s0);
    stage_scales<FMT, CB>(st + S::CODES, g + 8, s1);
    const int nblk = min(CB, nb - chunk * CB);
    // rows g and g + 8 share the swizzle; a stage's offset is a multiple of 128
    const uint32_t code0 = uint32_t(st - lsm) + lane_code;
    const unsigned char* xc[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) xc[j] = xrow[j] + chunk * (CB * 64);
    float d[NT][4];
    // fold: the sums so far take the scale of block b
    auto block = [&](int b, bool start, bool fold) {
      uint32_t q0[4], q1[4];
      levels<F::HALF>(*reinterpret_cast<const uint32_t*>(lsm + (code0 ^ (b << 4))), q0);
      levels<F::HALF>(*reinterpret_cast<const uint32_t*>(lsm + (code0 ^ (b << 4)) + 8 * S::ROW), q1);
      const uint32_t lo[4] = {q0[0], q1[0], q0[1], q1[1]}, hi[4] = {q0[2], q1[2], q0[3], q1[3]};
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint4 xv = *reinterpret_cast<const uint4*>(xc[j] + b * 64);
        if (start) mma16816(d[j], lo, xv.x, xv.y, 0.f, 0.f, 0.f, 0.f);
        else mma16816(d[j], lo, xv.x, xv.y, d[j][0], d[j][1], d[j][2], d[j][3]);
        mma16816(d[j], hi, xv.z, xv.w, d[j][0], d[j][1], d[j][2], d[j][3]);
        if (fold) {
          acc[j][0] = fmaf(s0[b], d[j][0], acc[j][0]);
          acc[j][1] = fmaf(s0[b], d[j][1], acc[j][1]);
          acc[j][2] = fmaf(s1[b], d[j][2], acc[j][2]);
          acc[j][3] = fmaf(s1[b], d[j][3], acc[j][3]);
        }
      }
    };
    if (nblk == CB) {
#pragma unroll
      for (int b = 0; b < CB; ++b) block(b, !F::G128 || (b & 3) == 0, !F::G128 || (b & 3) == 3);
    } else {
#pragma unroll
      for (int b = 0; b < CB - 1; ++b)
        if (b < nblk) block(b, !F::G128 || (b & 3) == 0, !F::G128 || (b & 3) == 3);
    }
    chunk += a.KG;
    if (chunk < a.chunks) continue;

    // ---------------------------------------------- the tile's epilogue
    const int bar = 1 + grp, bar_n = a.KG * 32;
    auto group_sync = [&]() {
      if (a.KG > 1) named_bar_sync(bar, bar_n);
      else __syncwarp();
    };
    if (!first_tile) group_sync();    // the previous tile's sums have been read
    first_tile = false;
    float* gp = spart + size_t(grp) * a.KG * 16 * TP;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float* p = gp + (kw * 16 + g) * TP + 8 * j + 2 * t;
      *reinterpret_cast<float2*>(p) = make_float2(acc[j][0], acc[j][1]);
      *reinterpret_cast<float2*>(p + 8 * TP) = make_float2(acc[j][2], acc[j][3]);
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;
    }
    group_sync();
    const int row0 = tile * 16, tid = kw * 32 + lane;
    auto sum_of = [&](int row, int n) {
      const float* p = gp + row * TP + n;
      float v = 0.f;
#pragma unroll 4
      for (int w = 0; w < a.KG; ++w) v += p[w * 16 * TP];
      v *= sinv[n];
      if (FMT == F_E32) v *= __ldg(a.row_scales + row0 + row);
      return v;
    };
    if (!a.gated) {
      for (int o = tid; o < 16 * nt; o += bar_n) {
        const int row = o & 15, n = o >> 4;
        if (row0 + row >= a.N) continue;
        float v = sum_of(row, n);
        if (a.bias) v += __ldg(a.bias + row0 + row);
        store_as(a.y, a.y_type, size_t(t0 + n) * a.N + row0 + row, v);
      }
    } else {
      for (int o = tid; o < 8 * nt; o += bar_n) {
        const int i = o & 7, n = o >> 3;
        if (row0 + 2 * i >= a.N) continue;
        const float gt = sum_of(2 * i, n), up = sum_of(2 * i + 1, n);
        store_as(a.y, a.y_type, size_t(t0 + n) * (a.N >> 1) + (row0 >> 1) + i, gt / (1.f + expf(-gt)) * up);
      }
    }
    chunk = kw;
    tile += step;
  }
  cp_async_wait<0>();
}

template <int FMT, int CB>
cudaError_t launch_fmt(const LinearArgs& a, int nt, int grid, size_t smem, cudaStream_t s) {
  auto kern = nt == 1 ? linear_kernel<1, FMT, CB> : nt == 2 ? linear_kernel<2, FMT, CB> : linear_kernel<4, FMT, CB>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid), dim3(kThreads), smem, s, a);
}

template <int CB>
cudaError_t launch_stage(int fmt, const LinearArgs& a, int nt, int grid, size_t smem, cudaStream_t s) {
  switch (fmt) {
    case F_H32: return launch_fmt<F_H32, CB>(a, nt, grid, smem, s);
    case F_H128: return launch_fmt<F_H128, CB>(a, nt, grid, smem, s);
    case F_E32: return launch_fmt<F_E32, CB>(a, nt, grid, smem, s);
    case F_H32_HALF: return launch_fmt<F_H32_HALF, CB>(a, nt, grid, smem, s);
    default: return launch_fmt<F_H128_HALF, CB>(a, nt, grid, smem, s);
  }
}

int groups_of_8(int tt) { return tt <= 8 ? 1 : tt <= 16 ? 2 : 4; }

// The most tokens (up to 32) whose activations fit beside a ring.
int most_tokens(int ring, int nb) {
  int most = 0;
  for (int tt = 1; tt <= 32; ++tt)
    if (linear_smem(ring, nb, tt, groups_of_8(tt)) <= kMaxSmem) most = tt;
  return most;
}

}  // namespace

cudaError_t launch_linear(const LinearCall& c, int num_sms, cudaStream_t s) {
  LinearArgs a{};
  a.codes = c.codes; a.scales = c.scales; a.row_scales = c.row_scales; a.bias = c.bias; a.x = c.x; a.y = c.y;
  a.N = c.rows; a.K = c.cols; a.T = c.T;
  a.nb = c.cols / 32;
  a.spr = c.cols / c.block;
  a.x_type = c.x_type; a.y_type = c.y_type; a.gated = c.gated;
  const int fmt = c.scale_fmt == 1 ? F_E32
                  : c.block == 128 ? (c.half_levels ? F_H128_HALF : F_H128)
                                   : (c.half_levels ? F_H32_HALF : F_H32);
  const int tiles = (a.N + 15) / 16;
  // the wide stage unless it costs a token slice or there is too little work
  // for every warp of the machine to fill one
  const int most4 = min(c.T, most_tokens(Stage<4>::RING, a.nb)), most8 = min(c.T, most_tokens(Stage<8>::RING, a.nb));
  const bool wide = most8 > 0 && (c.T + most8 - 1) / most8 == (c.T + most4 - 1) / most4 &&
                    size_t(tiles) * ((a.nb + 7) / 8) >= size_t(num_sms) * kWarps;
  const int CB = wide ? 8 : 4, most = wide ? most8 : most4;
  a.chunks = (a.nb + CB - 1) / CB;
  a.ny = (c.T + most - 1) / most;
  a.tt = (c.T + a.ny - 1) / a.ny;
  a.ny = (c.T + a.tt - 1) / a.tt;
  // Warps per row tile: the split that ends first.  In cycles, roughly, and
  // per narrow stage: an SM that is full delivers one every 60; a warp alone
  // takes 250; joining and storing a tile takes a warp 200, and the SM 20 for
  // each warp that joins.
  const int sms = max(1, num_sms / a.ny), per_sm = (tiles + sms - 1) / sms;
  int best = 0;
  for (int kg = 1; kg <= min(kWarps, a.chunks); ++kg) {
    const int gr = min(kWarps / kg, per_sm), w = CB / 4;
    const int rounds = (per_sm + gr - 1) / gr, stages = (a.chunks + kg - 1) / kg;
    const int cost = max(per_sm * (a.chunks * w * 60 + kg * 20), rounds * (stages * w * 250 + 200));
    if (best == 0 || cost < best) {
      best = cost;
      a.KG = kg;
      a.groups = gr;
    }
  }
  const int gx = min((tiles + a.groups - 1) / a.groups, sms);
  const int nt = groups_of_8(a.tt);
  const size_t smem = linear_smem(wide ? Stage<8>::RING : Stage<4>::RING, a.nb, a.tt, nt);
  return wide ? launch_stage<8>(fmt, a, nt, gx * a.ny, smem, s) : launch_stage<4>(fmt, a, nt, gx * a.ny, smem, s);
}

}  // namespace moe
