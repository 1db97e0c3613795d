// Packing into the microscaled 4-bit floating-point formats.
//
//   mx: e = max(floor(log2 amax) - 2, -127) per 32 k, scale byte e + 127, codes
//       e2m1(x 2^-e): the power of two that puts the largest value in [4, 8),
//       where 6 is the largest code (values above saturate).
//   nv: s = e4m3(min(amax / (6 g), 448)) per 16 k with the tensor scale g, codes
//       e2m1(x * (1 / (s g))); every operation rounded to float32.
//   Rounding to nearest, ties to even.  A block with a NaN or an infinity gets
//   the NaN scale (0xFF, 0x7F) and zero codes, so that products see NaN.
//
// Bound by HBM: x is read once, half a byte a value and the scales written.
#include <algorithm>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include "launch.cuh"
#include "fp4.cuh"
#include "igemm.h"
#include "overlap.cuh"
#include "pack_values.cuh"
#include "ptx.cuh"

namespace igemm {

// Eight codes, element 0 in the lowest nibble.
__device__ __forceinline__ uint32_t fp4_codes8(const float *y)
{
    uint32_t r;
    asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n\t"
        "mov.b32 %0, {b0, b1, b2, b3};\n\t}"
        : "=r"(r)
        : "f"(y[0]), "f"(y[1]), "f"(y[2]), "f"(y[3]), "f"(y[4]), "f"(y[5]), "f"(y[6]), "f"(y[7]));
    return r;
}

// nv: the factor 1 / (s g) of every scale byte (0: all codes zero), made once per
// block of threads; mx needs none.
template <bool NV>
struct Fp4Factors {
    float of[NV ? 128 : 1];
    __device__ void fill(float g)
    {
        if constexpr (NV) {
            for (int s = threadIdx.x + threadIdx.y * blockDim.x; s < 128; s += blockDim.x * blockDim.y) {
                // the byte's value: 2^(e - 7) (1 + f / 8), subnormals 2^-6 f / 8
                const float v = s >= 8 ? __uint_as_float(((s >> 3) + 120u) << 23 | static_cast<uint32_t>(s & 7) << 20)
                                       : static_cast<float>(s) * 0.001953125f;
                const float t = v * g;
                of[s] = t >= 1.17549435e-38f ? __frcp_rn(t) : 0.0f;
            }
            __syncthreads();
        }
    }
};

// The scale byte of a block whose largest magnitude is `amax` (bits: NaN sorts
// above infinity) and the factor that takes its values to codes (0: all
// codes zero).  g6: 6 g.
template <bool NV>
__device__ __forceinline__ uint8_t fp4_scale(uint32_t amax_bits, float g6, const Fp4Factors<NV> &factors, float &factor)
{
    const bool fine = amax_bits < 0x7F800000u;
    factor = 0.0f;
    if constexpr (!NV) {
        if (!fine) return 0xFF;
        if (amax_bits == 0) {
            factor = __uint_as_float(254u << 23);  // 2^127: the codes keep the zeros' signs
            return 0;
        }
        // floor(log2): the exponent field, or the leading bit of a subnormal
        const int lg = amax_bits >= 0x00800000u ? static_cast<int>(amax_bits >> 23) - 127
                                                : -118 - __clz(static_cast<int>(amax_bits));
        const int e = max(lg - 2, -127);
        factor = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
        return static_cast<uint8_t>(e + 127);
    } else {
        if (!fine) return 0x7F;
        const float q = fminf(__fdiv_rn(__uint_as_float(amax_bits), g6), 448.0f);
        uint16_t h;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(0.0f), "f"(q));
        factor = factors.of[h & 0x7F];
        return static_cast<uint8_t>(h & 0xFF);
    }
}

struct Fp4PackParams {
    int64_t ld;
    const int *index;
    const float *g;
    uint8_t *codes, *scales;
    int x_rows, rows, K, code_bytes, pitch;
};

// Row-major x: a thread per 16 k of a row (mx: two neighbouring lanes share a
// block's scale), so a warp reads and writes contiguous runs.  A block of threads
// is blockDim.x items (even) of blockDim.y rows; rows longer than that take
// several (blockIdx.y), and a thread goes down the rows, the next row's values and
// the index after that in flight.  Bound by HBM where the rows are read once (16384 x
// 8192: bfloat16 56 us, 6.0 TB/s; float32 90 us, 6.8 TB/s).
template <bool NV, class T, bool VEC>
__global__ void __launch_bounds__(256, VEC ? 5 : 4) pack_fp4_rows_kernel(const T *x, const Fp4PackParams p)
{
    overlap_wait();
    const int k = (blockIdx.y * blockDim.x + threadIdx.x) * 16;
    const bool in_row = k < 2 * p.code_bytes;
    const bool last = k / 8 + 2 == p.code_bytes / 4;  // of the row: it writes the padding
    const float g = NV && p.g ? *p.g : 1.0f;
    __shared__ Fp4Factors<NV> factors;
    factors.fill(g);
    const float g6 = 6.0f * g;
    const int step = gridDim.x * blockDim.y;
    // rows as unsigned: the last step past 2^31 does not wrap
    uint32_t row = blockIdx.x * blockDim.y + threadIdx.y;
    const uint32_t rows = static_cast<uint32_t>(p.rows);
    const auto source = [&](uint32_t r) {
        if (r >= rows) return -1;
        const int s = p.index ? p.index[r] : static_cast<int>(r);
        return s < p.x_rows ? s : -1;
    };
    Fp4Raw<T, VEC> raw;
    const auto load = [&](int src) {
        if (src >= 0 && in_row) raw.load(x + src * p.ld, k, p.K);
        else raw.zero();
    };
    load(source(row));
    int src = source(row + step);
    uint8_t *codes = p.codes + static_cast<int64_t>(row) * p.code_bytes + k / 2;
    uint8_t *scales = p.scales + static_cast<int64_t>(row) * p.pitch;
    const int64_t code_step = static_cast<int64_t>(step) * p.code_bytes, scale_step = static_cast<int64_t>(step) * p.pitch;
    // (the same count for every lane of a warp)
    for (; row - threadIdx.y < rows; row += step, codes += code_step, scales += scale_step) {
        float v[16];
        uint32_t amax = raw.unpack(v);
        load(src);
        src = source(row + 2 * step);
        if constexpr (!NV) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        if (!in_row || row >= rows) continue;
        float f;
        const uint8_t s = fp4_scale<NV>(amax, g6, factors, f);
        uint2 out = make_uint2(0, 0);
        if (amax < 0x7F800000u && f > 0.0f) {
#pragma unroll
            for (int i = 0; i < 16; i += 2) fp4_mul2(v[i], v[i + 1], f);
            out = make_uint2(fp4_codes8(v), fp4_codes8(v + 8));
        }
        *reinterpret_cast<uint2 *>(codes) = out;
        if (NV) {
            if (k < p.K) scales[k / 16] = s;
        } else if ((k & 16) == 0) {
            scales[k / 32] = s;
        }
        if (last)
            for (int b = (p.K + (NV ? 15 : 31)) / (NV ? 16 : 32); b < p.pitch; ++b) scales[b] = 0;
    }
    overlap_release();
}

// Transposed x [K, rows]: a CTA takes 32 R rows (R a lane, so loads run along x's
// rows; R = 2 for pairs of 16-bit values) by 256 k (32 per warp), and the packed rows
// go through shared memory to leave as runs of 128 bytes.  Bound by HBM (28672 x 8192
// float32: 158 us, 6.7 TB/s).
template <bool NV, class T, int R>
__global__ void __launch_bounds__(256) pack_fp4_transposed_kernel(const T *x, const Fp4PackParams p)
{
    static_assert(R == 1 || sizeof(T) == 2, "pairs of 16-bit values");
    overlap_wait();
    constexpr int kPerWarp = NV ? 2 : 1;  // scale bytes
    constexpr int kRows = 32 * R;
    __shared__ uint4 codes[kRows][9];     // (row pitch 144 bytes: no bank conflicts)
    __shared__ uint8_t scales[kRows][16];
    __shared__ Fp4Factors<NV> factors;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows;
    const int k0 = blockIdx.y * 256, k = k0 + 32 * warp;
    const float g = NV && p.g ? *p.g : 1.0f;
    factors.fill(g);
    const float g6 = 6.0f * g;
    float v[R][32];
    const T *src = x + static_cast<int64_t>(k) * p.ld + r0 + R * lane;
    if (r0 + R * lane + R <= p.rows && k + 32 <= p.K) {
        if constexpr (R == 2) {
            uint32_t raw[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) raw[i] = *reinterpret_cast<const uint32_t *>(src + i * p.ld);
#pragma unroll
            for (int i = 0; i < 32; ++i) fp4_floats<T>(raw[i], v[0][i], v[1][i]);
        } else {
            T raw[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) raw[i] = src[i * p.ld];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[0][i] = fp4_float(raw[i]);
        }
    } else {
#pragma unroll
        for (int q = 0; q < R; ++q)
#pragma unroll
            for (int i = 0; i < 32; ++i)
                v[q][i] = r0 + R * lane + q < p.rows && k + i < p.K ? fp4_float(src[i * p.ld + q]) : 0.0f;
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const int row = R * lane + q;
        uint32_t out[4] = {0, 0, 0, 0};
#pragma unroll
        for (int b = 0; b < kPerWarp; ++b) {
            constexpr int kBlock = 32 / kPerWarp;
            float *vb = v[q] + b * kBlock;
            uint32_t amax = 0;
#pragma unroll
            for (int i = 0; i < kBlock; ++i) amax = max(amax, __float_as_uint(vb[i]) & 0x7FFFFFFFu);
            float f = 0.0f;
            scales[row][warp * kPerWarp + b] = k + b * kBlock < p.K ? fp4_scale<NV>(amax, g6, factors, f) : 0;
            if (amax < 0x7F800000u && f > 0.0f) {
#pragma unroll
                for (int i = 0; i < kBlock; i += 2) fp4_mul2(vb[i], vb[i + 1], f);
#pragma unroll
                for (int i = 0; i < kBlock / 8; ++i) out[b * kBlock / 8 + i] = fp4_codes8(vb + 8 * i);
            }
        }
        codes[row][warp] = make_uint4(out[0], out[1], out[2], out[3]);
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < R; ++q) {
        const int r = (threadIdx.x >> 3) + 32 * q, c = threadIdx.x & 7;  // a row's 128 bytes from eight lanes
        const int at = k0 / 2 + 16 * c;
        if (r0 + r < p.rows && at < p.code_bytes)
            *reinterpret_cast<uint4 *>(p.codes + (r0 + r) * p.code_bytes + at) = codes[r][c];
    }
    for (int i = threadIdx.x; i < kRows * 8 * kPerWarp; i += 256) {
        const int r = i / (8 * kPerWarp), b = i % (8 * kPerWarp), at = blockIdx.y * 8 * kPerWarp + b;
        if (r0 + r < p.rows && at < p.pitch) p.scales[(r0 + r) * p.pitch + at] = scales[r][b];
    }
    overlap_release();
    // (mx: 256 k are half of 16 scale bytes) zeros from here up to the pitch
    if (blockIdx.y == gridDim.y - 1 && threadIdx.x < kRows && r0 + threadIdx.x < p.rows)
        for (int b = (blockIdx.y + 1) * 8 * kPerWarp; b < p.pitch; ++b) p.scales[(r0 + threadIdx.x) * p.pitch + b] = 0;
}

static_assert(IGEMM_FP4_MAX_K / 256 <= 65535, "the k axis fits in grid.y (256 k a block at least)");

template <bool NV, class T>
static int launch_pack_type(const Fp4PackCall &c, const Fp4PackParams &p, cudaStream_t stream)
{
    const T *x = static_cast<const T *>(c.x);
    if (c.transposed) {
        const int by = (c.K + 255) / 256;
        const auto launch = [&](auto kernel, int rows) {
            return launch_overlapped(kernel, dim3(static_cast<unsigned>((int64_t(c.rows) + rows - 1) / rows), by),
                                     dim3(256), 0, stream, x, p);
        };
        // pairs where every row of x starts on 4 bytes (16384 x 8192 bfloat16: 69 -> 56 us)
        if constexpr (sizeof(T) == 2)
            if (reinterpret_cast<uintptr_t>(x) % 4 == 0 && c.ld % 2 == 0)
                return launch(pack_fp4_transposed_kernel<NV, T, 2>, 64);
        return launch(pack_fp4_transposed_kernel<NV, T, 1>, 32);
    } else {
        const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && c.ld * sizeof(T) % 16 == 0;
        // a row's items in equal blocks of at most 256 threads, whole warps (short
        // rows: a power of two, several rows a warp), and as many rows as fit
        const int items = p.code_bytes / 8;
        const int chunks = (items + 255) / 256;
        int bx = ((items + chunks - 1) / chunks + 31) / 32 * 32;
        if (items <= 16)
            for (bx = 2; bx < items;) bx *= 2;
        const int by = std::max(1, 256 / bx);
        // blocks that are resident at once, fewer where the rows give one each
        const int64_t full = std::max<int64_t>(1, int64_t(sm_count()) * (vec ? 5 : 4) * std::max(1, 256 / (bx * by)) / chunks);
        const int64_t gx = std::min((int64_t(c.rows) + by - 1) / by, full);
        const dim3 grid(static_cast<unsigned>(gx), chunks), block(bx, by);
        const auto kernel = vec ? pack_fp4_rows_kernel<NV, T, true> : pack_fp4_rows_kernel<NV, T, false>;
        return launch_overlapped(kernel, grid, block, 0, stream, x, p);
    }
}

template <bool NV>
static int launch_pack_format(const Fp4PackCall &c, cudaStream_t stream)
{
    Fp4PackParams p{};
    p.ld = c.ld;
    p.index = c.index;
    p.g = c.tensor_scale;
    p.codes = c.codes;
    p.scales = c.scales;
    p.x_rows = c.x_rows;
    p.rows = c.rows;
    p.K = c.K;
    p.code_bytes = fp4_code_bytes(c.K);
    p.pitch = fp4_scale_pitch(c.K, NV);
    switch (c.x_type) {
    case 0: return launch_pack_type<NV, float>(c, p, stream);
    case 1: return launch_pack_type<NV, __nv_bfloat16>(c, p, stream);
    default: return launch_pack_type<NV, __half>(c, p, stream);
    }
}

// Packed rows copied to their places: zeros where the index is out of range.  A
// thread takes one 16-byte piece of four rows, a quarter of the rows apart, all in
// flight (four pieces in a row, each with its own division, took 64 instructions a
// piece: 17.9 us for 32768 rows of 2304 bytes against 15.6).  (The index is read for
// every quarter, the last row's where there is none: a branch around each of these loads
// takes the whole call from 22.8 to 24.1 us.)
__global__ void __launch_bounds__(256) fp4_copy_rows_kernel(const uint4 *codes, const uint4 *scales, const Fp4PackParams p)
{
    overlap_wait();
    const uint32_t cq = p.code_bytes / 16, per_row = cq + p.pitch / 16;
    const uint32_t rows = static_cast<uint32_t>(p.rows), quarter = (rows + 3) / 4;
    const uint32_t item = blockIdx.x * 256 + threadIdx.x;  // (fits: pack_once)
    const uint32_t row = item / per_row, j = item - row * per_row;
    if (row >= quarter) return;  // (an exit counts as a release)
    const bool code = j < cq;
    const int64_t pitch = code ? cq : per_row - cq;
    const uint4 *from = code ? codes + j : scales + (j - cq);
    uint4 *to = code ? reinterpret_cast<uint4 *>(p.codes) + j : reinterpret_cast<uint4 *>(p.scales) + (j - cq);
    int src[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) src[i] = p.index[min(row + i * quarter, rows - 1)];
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = make_uint4(0, 0, 0, 0);
        if (src[i] >= 0 && src[i] < p.x_rows) v[i] = from[src[i] * pitch];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t r = row + i * quarter;
        if (r < rows) to[r * pitch] = v[i];
    }
    overlap_release();
}

// Rows that are gathered twice or more on average are packed once, into a workspace,
// and copied from there, where that saves reading 32 MB of x at least: 32768 x 4096
// nvfp4 rows of 4096 take 45.0 -> 23.0 us (float32 84 -> 30), and 8192 x 4096 of 4096
// 13.5 -> 13.1; with 28 MB saved the GPU would still gain (4096 x 4096 of 512: 7.2 -> 5.3
// us), but a loop of calls is slower (7.4 -> 9.3) for a second launch and a workspace.
static bool pack_once(const Fp4PackCall &c)
{
    const int64_t pieces = fp4_code_bytes(c.K) / 16 + fp4_scale_pitch(c.K, c.nv) / 16;
    const int64_t saved = (int64_t(c.rows) - c.x_rows) * c.K * (c.x_type == 0 ? 4 : 2);
    return c.index && c.x_rows > 0 && c.rows / 2 >= c.x_rows && saved >= int64_t(1) << 25 &&
           c.rows * pieces <= 0xFFFFFFFFll - 1024;
}

int launch_fp4_pack(const Fp4PackCall &c, cudaStream_t stream)
{
    const auto launch = [&](const Fp4PackCall &call) {
        return call.nv ? launch_pack_format<true>(call, stream) : launch_pack_format<false>(call, stream);
    };
    if (!pack_once(c)) return launch(c);
    Fp4PackParams p{};
    p.index = c.index;
    p.codes = c.codes;
    p.scales = c.scales;
    p.x_rows = c.x_rows;
    p.rows = c.rows;
    p.code_bytes = fp4_code_bytes(c.K);
    p.pitch = fp4_scale_pitch(c.K, c.nv);
    const size_t code_bytes = size_t(c.x_rows) * p.code_bytes;
    void *ws = nullptr;
    if (workspace_alloc(&ws, code_bytes + size_t(c.x_rows) * p.pitch, stream) != kOk) {
        cudaGetLastError();  // no room for it: row by row
        return launch(c);
    }
    Fp4PackCall once = c;
    once.index = nullptr;
    once.rows = c.x_rows;
    once.codes = static_cast<uint8_t *>(ws);
    once.scales = once.codes + code_bytes;
    int rc = launch(once);
    if (rc == kOk) {
        const int64_t items = (int64_t(c.rows) + 3) / 4 * ((int64_t(p.code_bytes) + p.pitch) / 16);
        rc = launch_overlapped(fp4_copy_rows_kernel, dim3(static_cast<unsigned>((items + 255) / 256)), dim3(256), 0,
                               stream, reinterpret_cast<const uint4 *>(once.codes),
                               reinterpret_cast<const uint4 *>(once.scales), p);
    }
    if (workspace_free(ws, stream) != kOk) rc = kCudaError;
    return rc;
}

}  // namespace igemm
