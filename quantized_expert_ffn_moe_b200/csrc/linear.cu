// Products of few token rows with a packed 4-bit matrix: a plain linear layer
// and the gate/up half of a gated feed-forward block.
//
//   z[t][n] = rs_n * sum_b s_{n,b} * sum_{k in block b} (c_{n,k} - off) x[t][k]
//   linear: y[t][n] = z[t][n] (+ bias[n]);   gated: h[t][i] = silu(z[t][2i]) * z[t][2i+1]
//
// (c the stored code, off = 8 or 7.5, s the block's scale, rs the row scale of
// the fp8 format.)  Bound by the packed bytes, n * k / 2 plus the scales.
//
// A warp multiplies 16 rows at a time with the warp-level tensor instruction
// m16n8k16 (fp16 operands, fp32 accumulation), rows as M and up to 8 tokens as
// N, one 32-element block per two instructions, so that a block's sum comes
// out by itself and its scale enters fp32 with one multiply-add per row and
// token.  The instruction issues every 2 cycles per SM (measured); the HBM
// rate brings 16 rows x 16 codes every 5.5 cycles, so up to two groups of 8
// tokens run below the memory bound and dequantising is what must be cheap:
//  * A code is never converted.  Its bits, masked in place, are an fp16
//    subnormal: c * 2^-24 (mask 0x000f000f) or 16 c * 2^-24 (0x00f000f0), and
//    the tensor core takes subnormals exactly.  Eight codes cost four masks
//    and one shift.  The factor 16 is divided out of the activations of the
//    odd elements (a power of two, exact).
//  * The offset is not subtracted from the codes: the accumulator of a block
//    starts at -off * 2^-24 * sum_{k in b} x[t][k], computed once per call.
//  * The k order inside a block is free as long as both operands share it:
//    lane t of a row's quad takes the block's t-th 32-bit word, as stored.
// Activations become fp16 after the power of two that brings the row's largest
// magnitude into [2^13, 2^14): exact for every element within 2^-31 of that
// largest one, off by at most 2^-35 of it below (fp32 sums lose more).  A row
// with an infinity or a NaN gives NaN in all its outputs.
//
// Each warp streams its own 16 rows x 128 columns stages through a private
// ring of asynchronous copies (no block-wide barrier in the stream); the warps
// of a group split the columns of a row tile, so that even 2048 x 2048 spreads
// over 128 SMs, and join their fp32 sums through shared memory in a fixed
// order: the same inputs give the same bits.
#include "dense_internal.cuh"

namespace moe {

namespace {

constexpr int kWarps = 16;
constexpr int kThreads = kWarps * 32;
constexpr int kStages = 4;
constexpr int kChunk = 128;                                 // columns of a stage
constexpr int kCodeBytes = 16 * kChunk / 2;                 // 1 KB of codes
constexpr int kStageBytes = kCodeBytes + 128;               // + up to 16 x 4 fp16 scales
constexpr int kRingBytes = kWarps * kStages * kStageBytes;
constexpr size_t kMaxSmem = 232448;

// scale formats: fp16 per 32, fp16 per 128, E4M3 per 32 under a row scale
enum { F_H32 = 0, F_H128 = 1, F_E32 = 2 };

struct LinearArgs {
  const uint8_t* codes;
  const void* scales;
  const float* row_scales;
  const float* bias;
  const void* x;
  void* y;
  int N, K, T;          // matrix rows, columns, token rows
  int nb;               // 32-element blocks of a row
  int chunks;           // 128-column stages of a row
  int KG, groups;       // warps splitting a row tile's columns; row tiles in flight per CTA
  int ny, tt;           // token slices, tokens of a slice
  int x_type, y_type, gated, aligned;
  float off;
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

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Scales of a stage's four blocks of one row as floats, from the row's slot of
// 8 (fp16), 4 (E4M3) or 2 bytes (one fp16 for all four).
template <int FMT>
__device__ __forceinline__ void stage_scales(const unsigned char* sc, int row, float (&s)[4]) {
  if (FMT == F_H32) {
    const uint2 v = *reinterpret_cast<const uint2*>(sc + row * 8);
    const float2 a = __half22float2(u32_as_h2(v.x)), b = __half22float2(u32_as_h2(v.y));
    s[0] = a.x; s[1] = a.y; s[2] = b.x; s[3] = b.y;
  } else if (FMT == F_E32) {
    const uint32_t v = *reinterpret_cast<const uint32_t*>(sc + row * 4);
    uint32_t lo, hi;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi) : "r"(v));
    const float2 a = __half22float2(u32_as_h2(lo)), b = __half22float2(u32_as_h2(hi));
    s[0] = a.x; s[1] = a.y; s[2] = b.x; s[3] = b.y;
  } else {
    const float v = __half2float(*reinterpret_cast<const __half*>(sc + row * 2));
    s[0] = v; s[1] = v; s[2] = v; s[3] = v;
  }
}

// Shared memory: ring | x [nb][tt][4] 16-byte words | init [nb][8 NT] floats |
// partial sums [groups KG][16][8 NT] floats | inv [8 NT] floats | row maxima
// [tt][16] u32.
__host__ __device__ inline size_t linear_smem(int nb, int tt, int nt) {
  return size_t(kRingBytes) + size_t(nb) * tt * 64 + size_t(nb) * nt * 32 + size_t(kWarps) * 16 * 8 * nt * 4 +
         size_t(nt) * 32 + size_t(tt) * 64;
}

template <int NT, int FMT>
__global__ void __launch_bounds__(kThreads, 1) linear_kernel(const LinearArgs a) {
  extern __shared__ __align__(128) unsigned char lsm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int nb = a.nb, tt = a.tt;
  constexpr int TP = 8 * NT;
  unsigned char* sx = lsm + kRingBytes;
  float* sinit = reinterpret_cast<float*>(sx + size_t(nb) * tt * 64);
  float* spart = sinit + size_t(nb) * TP;
  float* sinv = spart + kWarps * 16 * TP;
  uint32_t* smax = reinterpret_cast<uint32_t*>(sinv + TP);

  const int slice = int(blockIdx.x % unsigned(a.ny)), cta = int(blockIdx.x / unsigned(a.ny));
  const int ctas = int(gridDim.x / unsigned(a.ny));
  const int t0 = slice * tt, nt = min(tt, a.T - t0);     // this CTA's tokens
  const int ntiles = (a.N + 15) >> 4;
  const int grp = warp / a.KG, kw = warp - grp * a.KG;
  const int first = cta * a.groups + grp, step = ctas * a.groups;
  const bool active = grp < a.groups;
  const int my_chunks = active && kw < a.chunks ? (a.chunks - kw + a.KG - 1) / a.KG : 0;
  const int my_tiles = active && first < ntiles ? (ntiles - first + step - 1) / step : 0;
  const int total = my_tiles * my_chunks;

  unsigned char* ring = lsm + warp * (kStages * kStageBytes);
  const size_t row_bytes = size_t(a.K) >> 1;
  constexpr int SPC = FMT == F_H128 ? 1 : 4;              // scales of a row in a stage
  constexpr int SB = FMT == F_E32 ? 1 : 2;                // bytes of a scale
  const int spr = FMT == F_H128 ? a.chunks : nb;          // scales of a row
  // scales that cannot be copied asynchronously (rows off a 4- or 8-byte
  // boundary, or one fp16 per stage) pass through registers: loaded with
  // their stage's codes, stored to its slot when the next stage is issued
  constexpr int PEND = (16 * SPC + 31) / 32;
  uint16_t pend[PEND];
  int pend_slot = -1;
  const bool direct = FMT != F_H128 && a.aligned;

  int it_tile = first, it_chunk = kw, issued = 0;
  auto flush_pending = [&]() {
    if (pend_slot < 0) return;
    unsigned char* sc = ring + pend_slot * kStageBytes + kCodeBytes;
#pragma unroll
    for (int i = 0; i < PEND; ++i) {
      const int e = i * 32 + lane;
      if (e < 16 * SPC) {
        if (SB == 2) *reinterpret_cast<uint16_t*>(sc + e * 2) = pend[i];
        else sc[e] = uint8_t(pend[i]);
      }
    }
    pend_slot = -1;
  };
  auto issue = [&]() {
    if (!direct) flush_pending();
    if (issued < total) {
      const int slot = issued % kStages;
      const uint32_t dst = smem_u32(ring) + slot * kStageBytes;
      const int row0 = it_tile * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = i * 8 + (lane >> 2), ch = lane & 3;
        if (it_chunk * 4 + ch < nb)
          cp_async16(dst + r * 64 + ((ch ^ ((r >> 1) & 3)) << 4),
                     a.codes + size_t(min(row0 + r, a.N - 1)) * row_bytes + size_t(it_chunk) * 64 + ch * 16);
      }
      if (direct) {
        if (lane < 16)
          cp_async_small<4 * SB>(dst + kCodeBytes + lane * (4 * SB),
                                 static_cast<const uint8_t*>(a.scales) +
                                     (size_t(min(row0 + lane, a.N - 1)) * spr + size_t(it_chunk) * 4) * SB);
      } else {
#pragma unroll
        for (int i = 0; i < PEND; ++i) {
          const int e = i * 32 + lane, r = e / SPC, b = it_chunk * SPC + e % SPC;
          pend[i] = 0;
          if (e < 16 * SPC && b < spr) {
            const size_t at = size_t(min(row0 + r, a.N - 1)) * spr + b;
            pend[i] = SB == 2 ? ld_stream2(static_cast<const uint16_t*>(a.scales) + at)
                              : uint16_t(__ldg(static_cast<const uint8_t*>(a.scales) + at));
          }
        }
        pend_slot = slot;
      }
      ++issued;
      it_chunk += a.KG;
      if (it_chunk >= a.chunks) { it_chunk = kw; it_tile += step; }
    }
    cp_async_commit();
  };
  // the weights do not depend on the previous kernel of the stream
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue();

  pdl_wait();
  pdl_launch_dependents();

  // ------------------------------------------------------ activations
  // A unit is (token, slice of its columns); with fewer tokens than warps a
  // token's columns are split over several warps.
  {
    const int sl = nt >= kWarps ? 1 : kWarps / nt;         // slices of a token
    const int units = nt * sl;
    const int K8 = a.K >> 3;                               // 16-byte words of a token row
    const int per = ((K8 + sl - 1) / sl + 3) & ~3;         // whole blocks per slice
    const uint16_t* xb = static_cast<const uint16_t*>(a.x) + size_t(t0) * a.K;
    for (int u = warp; u < units; u += kWarps) {
      const int n = u / sl, p = u % sl;
      const uint4* src = reinterpret_cast<const uint4*>(xb + size_t(n) * a.K);
      uint32_t m = 0;
      for (int w = p * per + lane; w < min(K8, (p + 1) * per); w += 32) {
        const uint4 v = __ldg(src + w);
        const uint32_t q[4] = {v.x & 0x7fff7fffu, v.y & 0x7fff7fffu, v.z & 0x7fff7fffu, v.w & 0x7fff7fffu};
#pragma unroll
        for (int i = 0; i < 4; ++i) m = max(m, max(q[i] & 0xffffu, q[i] >> 16));
      }
      m = __reduce_max_sync(0xffffffffu, m);
      if (lane == 0) smax[n * 16 + p] = m;
    }
    __syncthreads();
    for (int u = warp; u < units; u += kWarps) {
      const int n = u / sl, p = u % sl;
      uint32_t m = 0;
      for (int i = 0; i < sl; ++i) m = max(m, smax[n * 16 + i]);
      const bool bf = a.x_type == MOE_BF16;
      const bool finite = m < (bf ? 0x7f80u : 0x7c00u);
      const float top = bf ? __uint_as_float(m << 16) : __half2float(__ushort_as_half((unsigned short)m));
      int sh = 0;
      if (finite && top > 0.f) {
        int ex;
        frexpf(top, &ex);
        sh = min(max(14 - ex, -120), 120);
      }
      const float mul = ldexpf(1.f, sh);
      if (p == 0 && lane == 0) sinv[n] = finite ? ldexpf(1.f, -sh) : __int_as_float(0x7fc00000);
      const uint4* src = reinterpret_cast<const uint4*>(xb + size_t(n) * a.K);
      const int end = min(K8, (p + 1) * per);
      for (int w0 = p * per; w0 < end; w0 += 32) {
        const int w = w0 + lane;
        float f[8];
        if (w < end) {
          const uint4 v = __ldg(src + w);
          const uint32_t q[4] = {v.x, v.y, v.z, v.w};
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
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) f[i] = 0.f;
        }
        // element pairs (j, j + 4) as the masked code words hold them, the
        // odd ones over 16; their sum from the rounded values
        float sum = 0.f;
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float m2 = (j & 1) ? mul * 0.0625f : mul;
          const __half2 h = __floats2half2_rn(f[j] * m2, f[j + 4] * m2);
          o[j] = h2_as_u32(h);
          const float2 r = __half22float2(h);
          sum += (r.x + r.y) * ((j & 1) ? 16.f : 1.f);
        }
        sum += __shfl_xor_sync(0xffffffffu, sum, 1);
        sum += __shfl_xor_sync(0xffffffffu, sum, 2);
        if (w < end) {
          const int b = w >> 2;
          *reinterpret_cast<uint4*>(sx + (size_t(b) * tt + n) * 64 + (w & 3) * 16) = make_uint4(o[0], o[1], o[2], o[3]);
          if ((w & 3) == 0) sinit[size_t(b) * TP + n] = -a.off * 5.9604644775390625e-8f * sum;
        }
      }
    }
    __syncthreads();
  }
  if (total == 0) return;             // whole warps; a group's warps leave together

  // ------------------------------------------------------------ stream
  // this lane's words of the tokens 8 j + g (the last token's where there is
  // none: those columns are never stored) and its pair of initial sums
  const unsigned char* xrow[NT];
#pragma unroll
  for (int j = 0; j < NT; ++j) xrow[j] = sx + min(8 * j + g, nt - 1) * 64 + t * 16;
  const float* init0 = sinit + 2 * t;
  const int xstep = tt * 64;
  float acc[NT][4];
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[j][i] = 0.f;

  int tile = first, chunk = kw;
  bool first_tile = true;
  for (int it = 0; it < total; ++it) {
    __syncwarp();                     // every lane is done with the slot that is filled next
    issue();
    cp_async_wait<kStages - 1>();
    __syncwarp();
    const unsigned char* st = ring + (it % kStages) * kStageBytes;
    float s0[4], s1[4];
    stage_scales<FMT>(st + kCodeBytes, g, s0);
    stage_scales<FMT>(st + kCodeBytes, g + 8, s1);
    const int nblk = min(4, nb - chunk * 4);
    const unsigned char* code0 = st + g * 64 + t * 4;
    const int sw = (g >> 1) & 3;                          // rows g and g + 8 share the swizzle
    auto block = [&](int b) {
      const uint32_t w0 = *reinterpret_cast<const uint32_t*>(code0 + ((b ^ sw) << 4));
      const uint32_t w1 = *reinterpret_cast<const uint32_t*>(code0 + 512 + ((b ^ sw) << 4));
      const uint32_t v0 = w0 >> 8, v1 = w1 >> 8;
      const int bb = chunk * 4 + b;
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const uint4 xv = *reinterpret_cast<const uint4*>(xrow[j] + bb * xstep);
        const float2 iv = *reinterpret_cast<const float2*>(init0 + bb * TP + 8 * j);
        float d[4] = {iv.x, iv.y, iv.x, iv.y};
        mma16816(d, w0 & 0x000f000fu, w1 & 0x000f000fu, w0 & 0x00f000f0u, w1 & 0x00f000f0u, xv.x, xv.y);
        mma16816(d, v0 & 0x000f000fu, v1 & 0x000f000fu, v0 & 0x00f000f0u, v1 & 0x00f000f0u, xv.z, xv.w);
        acc[j][0] = fmaf(s0[b], d[0], acc[j][0]);
        acc[j][1] = fmaf(s0[b], d[1], acc[j][1]);
        acc[j][2] = fmaf(s1[b], d[2], acc[j][2]);
        acc[j][3] = fmaf(s1[b], d[3], acc[j][3]);
      }
    };
    if (nblk == 4) {
#pragma unroll
      for (int b = 0; b < 4; ++b) block(b);
    } else {
#pragma unroll
      for (int b = 0; b < 3; ++b)
        if (b < nblk) block(b);
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
      float v = 0.f;
      for (int w = 0; w < a.KG; ++w) v += gp[(w * 16 + row) * TP + n];
      v = v * 16777216.f * sinv[n];
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

template <int FMT>
cudaError_t launch_fmt(const LinearArgs& a, int nt, int grid, size_t smem, cudaStream_t s) {
  auto kern = nt == 1 ? linear_kernel<1, FMT> : nt == 2 ? linear_kernel<2, FMT> : linear_kernel<4, FMT>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem));
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(grid), dim3(kThreads), smem, s, a);
}

}  // namespace

cudaError_t launch_linear(const LinearCall& c, int num_sms, cudaStream_t s) {
  LinearArgs a{};
  a.codes = c.codes; a.scales = c.scales; a.row_scales = c.row_scales; a.bias = c.bias; a.x = c.x; a.y = c.y;
  a.N = c.rows; a.K = c.cols; a.T = c.T;
  a.nb = c.cols / 32;
  a.chunks = (c.cols + kChunk - 1) / kChunk;
  a.x_type = c.x_type; a.y_type = c.y_type; a.gated = c.gated;
  a.off = c.half_levels ? 7.5f : 8.f;
  a.aligned = a.nb % 4 == 0;          // a stage's scales of a row start on a 4- or 8-byte boundary
  // warps per row tile: as many as have columns to take, evenly
  const int per = (a.chunks + kWarps - 1) / kWarps;
  a.KG = (a.chunks + per - 1) / per;
  a.groups = kWarps / a.KG;
  // tokens of a slice: the most (up to 32) whose activations fit beside the ring
  int most = 1;
  for (int tt = 2; tt <= 32; ++tt) {
    const int nt = tt <= 8 ? 1 : tt <= 16 ? 2 : 4;
    if (linear_smem(a.nb, tt, nt) <= kMaxSmem) most = tt;
  }
  most = min(most, c.T);
  a.ny = (c.T + most - 1) / most;
  a.tt = (c.T + a.ny - 1) / a.ny;
  a.ny = (c.T + a.tt - 1) / a.tt;
  const int nt = a.tt <= 8 ? 1 : a.tt <= 16 ? 2 : 4;
  const size_t smem = linear_smem(a.nb, a.tt, nt);
  const int tiles = (a.N + 15) / 16;
  const int want = (tiles + a.groups - 1) / a.groups;
  const int gx = max(1, min(want, num_sms / a.ny));
  const int grid = gx * a.ny;
  if (c.scale_fmt == 1) return launch_fmt<F_E32>(a, nt, grid, smem, s);
  if (c.block == 128) return launch_fmt<F_H128>(a, nt, grid, smem, s);
  return launch_fmt<F_H32>(a, nt, grid, smem, s);
}

}  // namespace moe
