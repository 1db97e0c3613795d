// Packing into fp8 codes with one float32 scale per 128 k of a row, or per 128 rows
// and 128 k.
//
//   s = max(max|x| / F, 2^-126), F the format's largest value (448, 57344), and codes
//   fp8(x * (1 / s)); every operation rounded to float32, the codes to nearest, ties to
//   even, saturating.  A block with a NaN or an infinity gets a NaN scale and zero
//   codes, so that products see NaN.
//
// Bound by HBM: x is read once, a byte a value and the scales written.
#include <algorithm>
#include <math_constants.h>
#include "launch.cuh"
#include "bsfp8.cuh"
#include "igemm.h"
#include "overlap.cuh"
#include "pack_values.cuh"
#include "ptx.cuh"

namespace igemm {

struct Bsfp8PackParams {
    int64_t ld;
    const int *index;
    uint8_t *codes;
    float *scales;
    int x_rows, rows, K, code_bytes, pitch;
};

// The scale of a block whose largest magnitude is `amax` (bits: NaN sorts above
// infinity) and the factor that takes its values to codes (0: all codes zero).
template <int FMT>
__device__ __forceinline__ float bsfp8_scale(uint32_t amax_bits, float &factor)
{
    factor = 0.0f;
    if (amax_bits >= 0x7F800000u) return CUDART_NAN_F;
    const float s = fmaxf(__fdiv_rn(__uint_as_float(amax_bits), FMT == 0 ? 448.0f : 57344.0f), 1.17549435e-38f);
    factor = __frcp_rn(s);
    return s;
}

// Sixteen codes of v * f, element 0 in the lowest byte.
template <int FMT>
__device__ __forceinline__ uint4 bsfp8_codes16(float (&v)[16], float f)
{
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 16; i += 2) fp4_mul2(v[i], v[i + 1], f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint16_t lo, hi;
        if constexpr (FMT == 0) {
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[4 * i + 1]), "f"(v[4 * i]));
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[4 * i + 3]), "f"(v[4 * i + 2]));
        } else {
            asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(v[4 * i + 1]), "f"(v[4 * i]));
            asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(v[4 * i + 3]), "f"(v[4 * i + 2]));
        }
        w[i] = lo | static_cast<uint32_t>(hi) << 16;
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Row-major x, a scale per row and 128 k: a thread per 16 k of a row, eight
// neighbouring lanes share a block's scale.  A block of threads is blockDim.x items (a
// multiple of eight) of blockDim.y rows; rows longer than that take several
// (blockIdx.y), and a thread goes down the rows, the next row's values and the index
// after that in flight.  (4096 x 4096 bfloat16 from a cold cache: 11.1 us, 4.6 TB/s with
// the start of the launch.)
template <int FMT, class T, bool VEC>
__global__ void __launch_bounds__(256, VEC ? 5 : 4) pack_bsfp8_rows_kernel(const T *x, const Bsfp8PackParams p)
{
    overlap_wait();
    const int k = (blockIdx.y * blockDim.x + threadIdx.x) * 16;
    const bool in_row = k < p.code_bytes;
    const bool last = k + 16 == p.code_bytes;  // of the row: it writes the padding of the scales
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
    uint8_t *codes = p.codes + static_cast<int64_t>(row) * p.code_bytes + k;
    float *scales = p.scales + static_cast<int64_t>(row) * p.pitch;
    const int64_t code_step = static_cast<int64_t>(step) * p.code_bytes, scale_step = static_cast<int64_t>(step) * p.pitch;
    // (the same count for every lane of a warp)
    for (; row - threadIdx.y < rows; row += step, codes += code_step, scales += scale_step) {
        float v[16];
        uint32_t amax = raw.unpack(v);
        load(src);
        src = source(row + 2 * step);
#pragma unroll
        for (int d = 1; d < 8; d *= 2) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, d));
        if (!in_row || row >= rows) continue;
        float f;
        const float s = bsfp8_scale<FMT>(amax, f);
        *reinterpret_cast<uint4 *>(codes) = f > 0.0f ? bsfp8_codes16<FMT>(v, f) : make_uint4(0, 0, 0, 0);
        if ((k & 127) == 0) scales[k / 128] = s;
        if (last)
            for (int b = k / 128 + 1; b < p.pitch; ++b) scales[b] = 0.0f;
    }
    overlap_release();
}

// The largest of the block's values (bits), the same in every thread.
__device__ __forceinline__ uint32_t bsfp8_block_max(uint32_t amax, uint32_t (&part)[8])
{
    amax = __reduce_max_sync(0xffffffffu, amax);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = amax;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 8; ++i) amax = max(amax, part[i]);
    return amax;
}

// Zeros after a row's last scale (the CTA of its last block writes them).
__device__ __forceinline__ void bsfp8_pad_scales(const Bsfp8PackParams &p, float *scales, int b)
{
    if (b == gridDim.y - 1)
        for (int i = b + 1; i < p.pitch; ++i) scales[i] = 0.0f;
}

// Row-major x, a scale per 128 rows and 128 k: a CTA per such tile, eight lanes a row
// and four rows a thread, held in registers as they were read until the tile's largest
// is known (one reading of x; a second one would be half as much traffic again).  (28672 x
// 8192: float32 177 us, 6.6 TB/s, bfloat16 106, 6.6; 4096 x 4096 bfloat16 10.2.)
template <int FMT, class T, bool VEC>
__global__ void __launch_bounds__(256) pack_bsfp8_tiles_kernel(const T *x, const Bsfp8PackParams p)
{
    __shared__ uint32_t part[8];
    overlap_wait();
    const int k = blockIdx.y * 128 + (threadIdx.x & 7) * 16;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * 128 + (threadIdx.x >> 3);
    Fp4Raw<T, VEC> raw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 32 * i;
        if (r < p.rows && k < p.K) raw[i].load(x + r * p.ld, k, p.K);
        else raw[i].zero();
    }
    uint32_t amax = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) amax = max(amax, raw[i].largest());
    amax = bsfp8_block_max(amax, part);
    float f;
    const float s = bsfp8_scale<FMT>(amax, f);
    if (threadIdx.x == 0) {
        float *to = p.scales + static_cast<int64_t>(blockIdx.x) * p.pitch;
        to[blockIdx.y] = s;
        bsfp8_pad_scales(p, to, blockIdx.y);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int64_t r = r0 + 32 * i;
        if (r >= p.rows || k >= p.code_bytes) continue;
        float v[16];
        raw[i].values(v);
        *reinterpret_cast<uint4 *>(p.codes + r * p.code_bytes + k) =
            f > 0.0f ? bsfp8_codes16<FMT>(v, f) : make_uint4(0, 0, 0, 0);
    }
    overlap_release();
}

// Transposed x [K, rows]: a CTA takes 128 k (16 per warp) by P times 32 R rows (R a
// lane, so loads run along x's rows; R = 2 for pairs of 16-bit values), held in
// registers until the largest of each row, or (TILE) of 128 rows, is known.  The codes
// go through shared memory to leave as runs of 128 bytes.  (28672 x 8192, a scale
// per 128 x 128: float32 189 us, 6.2 TB/s, bfloat16 109, 6.5; a scale per row 176, 6.7, and 127,
// 5.6.)
template <int FMT, class T, int R, bool TILE>
__global__ void __launch_bounds__(256) pack_bsfp8_transposed_kernel(const T *x, const Bsfp8PackParams p)
{
    static_assert(R == 1 || sizeof(T) == 2, "pairs of 16-bit values");
    constexpr int P = TILE ? 4 / R : 1, kRows = 32 * R * P;
    __shared__ uint4 codes[kRows][9];  // (row pitch 144 bytes)
    __shared__ uint32_t part[8];
    __shared__ uint32_t largest[TILE ? 1 : 8][TILE ? 1 : kRows];
    overlap_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * kRows;
    const int k = blockIdx.y * 128 + 16 * warp;
    uint32_t raw[P][16];  // a float32, or R 16-bit values
    uint32_t amax[R];
#pragma unroll
    for (int q = 0; q < R; ++q) amax[q] = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const int64_t r = r0 + 32 * R * i + R * lane;
        const T *src = x + static_cast<int64_t>(k) * p.ld + r;
        const bool whole = r + R <= p.rows && k + 16 <= p.K;
#pragma unroll
        for (int j = 0; j < 16; ++j) {
            uint32_t w = 0;
            if (whole) {
                if constexpr (sizeof(T) == 4 || R == 2) w = *reinterpret_cast<const uint32_t *>(src + j * p.ld);
                else w = *reinterpret_cast<const uint16_t *>(src + j * p.ld);
            } else if (k + j < p.K) {
#pragma unroll
                for (int q = 0; q < R; ++q)
                    if (r + q < p.rows) {
                        if constexpr (sizeof(T) == 4) w = *reinterpret_cast<const uint32_t *>(src + j * p.ld);
                        else w |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t *>(src + j * p.ld + q)) << (16 * q);
                    }
            }
            raw[i][j] = w;
        }
    }
    const auto value = [&](int i, int j, int q) {
        if constexpr (sizeof(T) == 4) {
            return __uint_as_float(raw[i][j]);
        } else {
            float lo, hi;
            fp4_floats<T>(raw[i][j], lo, hi);
            return q ? hi : lo;
        }
    };
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int j = 0; j < 16; ++j)
#pragma unroll
            for (int q = 0; q < R; ++q) amax[q] = max(amax[q], __float_as_uint(value(i, j, q)) & 0x7FFFFFFFu);
    float f[R];
    if constexpr (TILE) {
        uint32_t all = amax[0];
        if constexpr (R == 2) all = max(all, amax[1]);
        all = bsfp8_block_max(all, part);
        const float s = bsfp8_scale<FMT>(all, f[0]);
        if constexpr (R == 2) f[1] = f[0];
        if (threadIdx.x == 0) {
            float *to = p.scales + static_cast<int64_t>(blockIdx.x) * p.pitch;
            to[blockIdx.y] = s;
            bsfp8_pad_scales(p, to, blockIdx.y);
        }
    } else {
#pragma unroll
        for (int q = 0; q < R; ++q) largest[warp][R * lane + q] = amax[q];
        __syncthreads();
#pragma unroll
        for (int q = 0; q < R; ++q) {
            const int row = R * lane + q;
#pragma unroll
            for (int w = 0; w < 8; ++w) amax[q] = max(amax[q], largest[w][row]);
            const float s = bsfp8_scale<FMT>(amax[q], f[q]);
            if (warp == 0 && r0 + row < p.rows) {
                float *to = p.scales + (r0 + row) * p.pitch;
                to[blockIdx.y] = s;
                bsfp8_pad_scales(p, to, blockIdx.y);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
        for (int q = 0; q < R; ++q) {
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = value(i, j, q);
            codes[32 * R * i + R * lane + q][warp] =
                f[q] > 0.0f ? bsfp8_codes16<FMT>(v, f[q]) : make_uint4(0, 0, 0, 0);
        }
    __syncthreads();
    const int c = threadIdx.x & 7, at = blockIdx.y * 128 + 16 * c;  // a row's 128 bytes from eight lanes
#pragma unroll
    for (int r = threadIdx.x >> 3; r < kRows; r += 32)
        if (r0 + r < p.rows && at < p.code_bytes)
            *reinterpret_cast<uint4 *>(p.codes + (r0 + r) * p.code_bytes + at) = codes[r][c];
    overlap_release();
}

static_assert(IGEMM_BSFP8_MAX_K / 128 <= 65535, "the k axis fits in grid.y (128 k a block at least)");

template <int FMT, class T>
static int launch_pack_type(const Bsfp8PackCall &c, const Bsfp8PackParams &p, cudaStream_t stream)
{
    const T *x = static_cast<const T *>(c.x);
    const unsigned blocks = static_cast<unsigned>((c.K + 127) / 128);
    if (c.transposed) {
        const auto launch = [&](auto kernel, int rows) {
            return launch_overlapped(kernel, dim3(static_cast<unsigned>((int64_t(c.rows) + rows - 1) / rows), blocks),
                                     dim3(256), 0, stream, x, p);
        };
        // pairs where every row of x starts on 4 bytes
        if constexpr (sizeof(T) == 2)
            if (reinterpret_cast<uintptr_t>(x) % 4 == 0 && c.ld % 2 == 0)
                return c.tile_rows == 1 ? launch(pack_bsfp8_transposed_kernel<FMT, T, 2, false>, 64)
                                        : launch(pack_bsfp8_transposed_kernel<FMT, T, 2, true>, 128);
        return c.tile_rows == 1 ? launch(pack_bsfp8_transposed_kernel<FMT, T, 1, false>, 32)
                                : launch(pack_bsfp8_transposed_kernel<FMT, T, 1, true>, 128);
    }
    const bool vec = reinterpret_cast<uintptr_t>(x) % 16 == 0 && c.ld * sizeof(T) % 16 == 0;
    if (c.tile_rows > 1) {
        const dim3 grid(static_cast<unsigned>((int64_t(c.rows) + 127) / 128), blocks);
        return launch_overlapped(vec ? pack_bsfp8_tiles_kernel<FMT, T, true> : pack_bsfp8_tiles_kernel<FMT, T, false>,
                                 grid, dim3(256), 0, stream, x, p);
    }
    // a row's items in equal blocks of at most 256 threads, whole warps (short rows: a
    // power of two, several rows a warp), and as many rows as fit
    const int items = p.code_bytes / 16;
    const int chunks = (items + 255) / 256;
    int bx = ((items + chunks - 1) / chunks + 31) / 32 * 32;
    if (items <= 16)
        for (bx = 8; bx < items;) bx *= 2;
    const int by = std::max(1, 256 / bx);
    // blocks that are resident at once, fewer where the rows give one each
    const int64_t full = std::max<int64_t>(1, int64_t(sm_count()) * (vec ? 5 : 4) * std::max(1, 256 / (bx * by)) / chunks);
    const int64_t gx = std::min((int64_t(c.rows) + by - 1) / by, full);
    return launch_overlapped(vec ? pack_bsfp8_rows_kernel<FMT, T, true> : pack_bsfp8_rows_kernel<FMT, T, false>,
                             dim3(static_cast<unsigned>(gx), chunks), dim3(bx, by), 0, stream, x, p);
}

template <int FMT>
static int launch_pack_format(const Bsfp8PackCall &c, cudaStream_t stream)
{
    Bsfp8PackParams p{};
    p.ld = c.ld;
    p.index = c.index;
    p.codes = c.codes;
    p.scales = c.scales;
    p.x_rows = c.x_rows;
    p.rows = c.rows;
    p.K = c.K;
    p.code_bytes = bsfp8_code_bytes(c.K);
    p.pitch = bsfp8_scale_pitch(c.K);
    switch (c.x_type) {
    case 0: return launch_pack_type<FMT, float>(c, p, stream);
    case 1: return launch_pack_type<FMT, __nv_bfloat16>(c, p, stream);
    default: return launch_pack_type<FMT, __half>(c, p, stream);
    }
}

// Packed rows copied to their places; where the index is out of range, a row of zeros.
// A thread takes one 16-byte piece of four rows, a quarter of the rows apart, all in flight.
// (32768 rows of 4096 out of 4096, 138 MB written: 36.0 us for both launches, with two or eight
// rows a thread 38.1 and 40.4, by bulk copies through shared memory 35.5.  With what is written
// the first to leave L2, so that the packed rows stay, 32.8; a product that reads the
// copies next takes as long as before.)
__global__ void __launch_bounds__(256) bsfp8_copy_rows_kernel(const uint4 *codes, const uint4 *scales, const Bsfp8PackParams p)
{
    overlap_wait();
    const uint32_t cq = p.code_bytes / 16, per_row = cq + p.pitch / 4;
    const uint32_t rows = static_cast<uint32_t>(p.rows), quarter = (rows + 3) / 4;
    const uint32_t item = blockIdx.x * 256 + threadIdx.x;  // (fits: pack_once)
    const uint32_t row = item / per_row, j = item - row * per_row;
    if (row >= quarter) return;  // (an exit counts as a release)
    const bool code = j < cq;
    const int64_t pitch = code ? cq : per_row - cq;
    const uint4 *from = code ? codes + j : scales + (j - cq);
    uint4 *to = code ? reinterpret_cast<uint4 *>(p.codes) + j : reinterpret_cast<uint4 *>(p.scales) + (j - cq);
    uint4 zeros = make_uint4(0, 0, 0, 0);
    if (!code) {  // (the scale of a block of zeros, 2^-126)
        const int left = (p.K + 127) / 128 - 4 * static_cast<int>(j - cq);
        constexpr uint32_t kLeast = 0x00800000u;
        zeros = make_uint4(left > 0 ? kLeast : 0, left > 1 ? kLeast : 0, left > 2 ? kLeast : 0, left > 3 ? kLeast : 0);
    }
    int src[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) src[i] = p.index[min(row + i * quarter, rows - 1)];
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = zeros;
        if (src[i] >= 0 && src[i] < p.x_rows) v[i] = from[src[i] * pitch];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t r = row + i * quarter;
        if (r < rows) __stcs(to + r * pitch, v[i]);
    }
    overlap_release();
}

// Rows that are gathered twice or more on average are packed once, into a workspace,
// and copied from there, where that saves reading 32 MB of x at least.  (32768 rows of 4096
// bfloat16 out of 4096: 32.8 us so, 50 row by row; a second launch costs 4.)
static bool pack_once(const Bsfp8PackCall &c)
{
    const int64_t pieces = bsfp8_code_bytes(c.K) / 16 + bsfp8_scale_pitch(c.K) / 4;
    const int64_t saved = (int64_t(c.rows) - c.x_rows) * c.K * (c.x_type == 0 ? 4 : 2);
    return c.index && c.x_rows > 0 && c.rows / 2 >= c.x_rows && saved >= int64_t(1) << 25 &&
           c.rows * pieces <= 0xFFFFFFFFll - 1024;
}

int launch_bsfp8_pack(const Bsfp8PackCall &c, cudaStream_t stream)
{
    const auto launch = [&](const Bsfp8PackCall &call) {
        return call.format == 0 ? launch_pack_format<0>(call, stream) : launch_pack_format<1>(call, stream);
    };
    if (!pack_once(c)) return launch(c);
    Bsfp8PackParams p{};
    p.index = c.index;
    p.codes = c.codes;
    p.scales = c.scales;
    p.x_rows = c.x_rows;
    p.rows = c.rows;
    p.K = c.K;
    p.code_bytes = bsfp8_code_bytes(c.K);
    p.pitch = bsfp8_scale_pitch(c.K);
    const size_t code_bytes = size_t(c.x_rows) * p.code_bytes;
    void *ws = nullptr;
    if (workspace_alloc(&ws, code_bytes + size_t(c.x_rows) * p.pitch * 4, stream) != kOk) {
        cudaGetLastError();  // no room for it: row by row
        return launch(c);
    }
    Bsfp8PackCall once = c;
    once.index = nullptr;
    once.rows = c.x_rows;
    once.codes = static_cast<uint8_t *>(ws);
    once.scales = reinterpret_cast<float *>(once.codes + code_bytes);
    int rc = launch(once);
    if (rc == kOk) {
        const int64_t items = (int64_t(c.rows) + 3) / 4 * (int64_t(p.code_bytes) / 16 + p.pitch / 4);
        rc = launch_overlapped(bsfp8_copy_rows_kernel, dim3(static_cast<unsigned>((items + 255) / 256)), dim3(256), 0,
                               stream, reinterpret_cast<const uint4 *>(once.codes),
                               reinterpret_cast<const uint4 *>(once.scales), p);
    }
    if (workspace_free(ws, stream) != kOk) rc = kCudaError;
    return rc;
}

}  // namespace igemm
