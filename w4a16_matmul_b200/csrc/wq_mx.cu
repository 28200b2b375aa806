// wq_mx.cu -- MXFP4 quantisation and reconstruction: the OCP microscaling format of 4-bit
// floating point, blocks of 32 consecutive values of a row with one power-of-two scale.
//
//   value = level(code) * 2^(s - 127),   level = 0, 1/2, 1, 3/2, 2, 3, 4, 6 by the code's low
//   three bits (E2M1: two exponent bits, one mantissa bit), negative when its bit 3 is set.
//
// The scale of a block is the power of two that brings its largest magnitude into [4, 8):
// s - 127 = floor(log2 amax) - 2, so s = max(E - 2, 0) with E the biased exponent field of
// amax (8 bits in bf16 and fp32 alike; zero and subnormal maxima have E = 0). Multiplying a
// value by 2^(127 - s) is exact (or underflows towards a value that codes to 0 anyway), and
// the conversion to E2M1 rounds once: to nearest, ties to the even code, 6 at most.
//
// Both kernels are HBM streams: a thread owns 8 consecutive values (a quarter of a block),
// its loads and stores are 128 bits wide, and a warp's accesses are contiguous.
// Measured at 8192 x 28672 bf16, 4.5 bytes a value with q: 164 us, 6.48 TB/s, what a copy reaches;
// its reconstruction, 2.5 bytes a value: 90 us, 6.6 TB/s.
#include "wq_internal.cuh"

namespace wq {
namespace {

constexpr int kThreads = 256;

// One trip a thread, the whole array in one grid: blocks that come and go keep loads and stores
// of the stream mixed (8192 x 28672 bf16 with q: 164 us; 8 resident blocks an SM in a loop: 200 us).
int stream_grid(int64_t items) {
    const int64_t blocks = (items + kThreads - 1) / kThreads;
    return (int)(blocks < 1 ? 1 : blocks > 0x7FFFFFFF ? 0x7FFFFFFF : blocks);
}

// One chunk of 8 values as loaded: 4 words of bf16 pairs, or 8 words of fp32.
template <bool F32>
struct Chunk {
    uint32_t w[F32 ? 8 : 4];
};

template <bool F32>
__device__ __forceinline__ Chunk<F32> load_chunk(const void* x, int64_t c, bool live) {
    Chunk<F32> r;
    if constexpr (F32) {
        // two 128-bit loads: addresses are multiples of 16 bytes, no more. With both halves of a
        // sector from one L1 line they are as fast as one 256-bit load on an address that allows it
        // (8192 x 14336 with q: 149 us both; 157 without L1 allocation)
        const uint4* p = (const uint4*)x + 2 * c;
        const uint4 a = live ? ldg_v4(p) : make_uint4(0, 0, 0, 0), b = live ? ldg_v4(p + 1) : make_uint4(0, 0, 0, 0);
        r.w[0] = a.x; r.w[1] = a.y; r.w[2] = a.z; r.w[3] = a.w;
        r.w[4] = b.x; r.w[5] = b.y; r.w[6] = b.z; r.w[7] = b.w;
    } else {
        const uint4 v = live ? ldg_nc_v4((const uint4*)x + c) : make_uint4(0, 0, 0, 0);
        r.w[0] = v.x; r.w[1] = v.y; r.w[2] = v.z; r.w[3] = v.w;
    }
    return r;
}

// Quantises the chunk c of the calling thread (four consecutive lanes hold one block), stores
// what was asked for and returns the scale byte. I: the index type of chunks.
template <bool F32, typename I>
__device__ __forceinline__ uint32_t quantise_chunk(const Chunk<F32>& ch, bool live, I c, uint2* __restrict__ codes,
                                                   uint32_t* __restrict__ packed, void* __restrict__ q) {
    // the block's largest magnitude as bits: their order is the values' order, with the
    // infinities and then the NaNs on top
    uint32_t top;
    float v[8];
    if constexpr (F32) {
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            top = max(top, ch.w[i] & 0x7FFFFFFFu);
            v[i] = __uint_as_float(ch.w[i]);
        }
    } else {
        const uint32_t m = max_u16x2(max_u16x2(ch.w[0] & 0x7FFF7FFFu, ch.w[1] & 0x7FFF7FFFu),
                                     max_u16x2(ch.w[2] & 0x7FFF7FFFu, ch.w[3] & 0x7FFF7FFFu));
        top = max(m << 16, m & 0xFFFF0000u);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(ch.w[i] << 16);
            v[2 * i + 1] = __uint_as_float(ch.w[i] & 0xFFFF0000u);
        }
    }
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const uint32_t s = mx_scale_byte(top >> 23);
    const bool bad = s == 255;                                 // a NaN or an infinity in the block
    const float inv = mx_inverse_scale(s);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= inv;
    const uint32_t p = bad ? 0u : e2m1x8(v);
    if (!live) return s;
    if (packed) packed[c] = p;
    if (codes) {
        const uint32_t e = p & 0x0F0F0F0Fu, o = (p >> 4) & 0x0F0F0F0Fu;
        codes[c] = make_uint2(prmt(e, o, 0x5140u), prmt(e, o, 0x7362u));
    }
    if (q) {
        uint32_t o[4];
        mx4_word(p, o);
        const uint32_t sc = mx_scale_pair(s);
#pragma unroll
        for (int i = 0; i < 4; ++i) o[i] = bf16x2_fma(o[i], sc, 0x80008000u);   // exact: 2 significant bits
        if constexpr (F32) {
            uint32_t f[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) { f[2 * i] = o[i] << 16; f[2 * i + 1] = o[i] & 0xFFFF0000u; }
            uint4* qc = (uint4*)q + 2 * (int64_t)c;
            stg_cs_v4(qc, make_uint4(f[0], f[1], f[2], f[3]));
            stg_cs_v4(qc + 1, make_uint4(f[4], f[5], f[6], f[7]));
        } else {
            stg_cs_v4((uint4*)q + c, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
    return s;
}

template <bool F32, typename I>
__global__ void __launch_bounds__(kThreads)
quantize_mxfp4_kernel(const void* __restrict__ x, I n_chunks, uint32_t kb, uint32_t pitch,
                      uint8_t* __restrict__ scale, uint2* __restrict__ codes, uint32_t* __restrict__ packed,
                      void* __restrict__ q, bool early) {
    constexpr int U = 2;
    constexpr uint32_t PER = 8 * U;                            // blocks of a warp's trip, consecutive
    // in front of a product (which waits before it reads what this writes): it may start. Not for
    // a caller's own quantisation: an overlapped GEMV plan two launches later would load weights
    // that are still being written here.
    if (early) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const I stride = (I)gridDim.x * blockDim.x * U;
    const I lane = threadIdx.x & 31;
    // a warp covers U consecutive runs of 32 chunks; a block never straddles n_chunks
    for (I c0 = ((I)blockIdx.x * blockDim.x + (threadIdx.x & ~31u)) * U; c0 < n_chunks; c0 += stride) {
        Chunk<F32> v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const I c = c0 + 32 * u + lane;
            v[u] = load_chunk<F32>(x, (int64_t)c, c < n_chunks);
        }
        uint32_t sb = 0;                                       // byte u: the scale of this lane's block of run u
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const I c = c0 + 32 * u + lane;
            sb |= quantise_chunk<F32, I>(v[u], c < n_chunks, c, codes, packed, q) << (8 * u);
        }
        if (scale) {
            // the trip's scale bytes lie side by side: lane i stores that of block i (run i / 8, lanes
            // 4 (i % 8) ..), so that one store covers them
            sb = __shfl_sync(0xFFFFFFFFu, sb, 4 * ((uint32_t)lane & 7)) >> (8 * ((uint32_t)lane >> 3));
            const I b = c0 / 4 + lane;
            if (lane < PER && b < n_chunks / 4) {
                if (pitch == kb) {
                    scale[b] = (uint8_t)sb;
                } else {
                    const I row = b / kb;
                    const uint32_t col = (uint32_t)(b - row * kb);
                    uint8_t* sr = scale + (int64_t)row * pitch;
                    sr[col] = (uint8_t)sb;
                    if (col == kb - 1)                         // the padding of the row's scales
                        for (uint32_t i = kb; i < pitch; ++i) sr[i] = 0;
                }
            }
        }
    }
}

// bf16(level * 2^(s - 127)): one packed word (8 codes) a thread and trip.
template <typename I>
__global__ void __launch_bounds__(kThreads)
dequant_mxfp4_kernel(const uint32_t* __restrict__ packed, const uint8_t* __restrict__ scale, I n_words, uint32_t kb,
                     uint32_t pitch, uint4* __restrict__ out) {
    constexpr int U = 4;
    const I lane = threadIdx.x & 31;
    const I stride = (I)gridDim.x * blockDim.x * U;
    for (I base = ((I)blockIdx.x * blockDim.x + (threadIdx.x & ~31u)) * U; base < n_words; base += stride) {
        uint32_t p[U], s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const I i = base + 32 * u + lane;
            p[u] = s[u] = 0;
            if (i < n_words) {
                p[u] = __ldg(packed + i);
                const I b = i >> 2, row = pitch == kb ? 0 : b / kb;
                s[u] = __ldg(scale + (int64_t)b + (int64_t)row * (pitch - kb));
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const I i = base + 32 * u + lane;
            if (i >= n_words) break;
            uint32_t o[4];
            mx4_word(p[u], o);
            const uint32_t sc = mx_scale_pair(s[u]);
#pragma unroll
            for (int j = 0; j < 4; ++j) o[j] = bf16x2_fma(o[j], sc, 0x80008000u);
            stg_cs_v4(out + i, make_uint4(o[0], o[1], o[2], o[3]));
        }
    }
}

}  // namespace

wq_status launch_quantize_mxfp4(const void* x, int dtype, int64_t n, int64_t k, uint8_t* scale, uint8_t* codes,
                                uint8_t* packed, void* q, bool early, cudaStream_t s) {
    const int64_t chunks = n * k / 8;
    constexpr int U = 2;
    const int grid = stream_grid((chunks + U - 1) / U);
    const uint32_t kb = (uint32_t)(k / 32), pitch = (uint32_t)mx_pitch(k);
    // 32-bit chunk indices while the last trip's c0 + stride stays below 2^32
    const bool narrow = chunks + (int64_t)grid * kThreads * U < (int64_t)1 << 32;
#define WQ_MXQ(F32, I)                                                                                     \
    quantize_mxfp4_kernel<F32, I><<<grid, kThreads, 0, s>>>(x, (I)chunks, kb, pitch, scale, (uint2*)codes, \
                                                            (uint32_t*)packed, q, early)
    if (dtype == WQ_F32) {
        if (narrow) WQ_MXQ(true, uint32_t); else WQ_MXQ(true, uint64_t);
    } else {
        if (narrow) WQ_MXQ(false, uint32_t); else WQ_MXQ(false, uint64_t);
    }
#undef WQ_MXQ
    return check_launch("quantize_mxfp4");
}

wq_status launch_dequant_mxfp4(const wq_weight& w, uint16_t* out, cudaStream_t s) {
    const int64_t words = w.n * w.k / 8;
    const int grid = stream_grid((words + 3) / 4);
    const uint32_t kb = (uint32_t)(w.k / 32), pitch = (uint32_t)mx_pitch(w.k);
    if (words + (int64_t)grid * kThreads * 4 < (int64_t)1 << 32)
        dequant_mxfp4_kernel<uint32_t><<<grid, kThreads, 0, s>>>((const uint32_t*)w.packed, (const uint8_t*)w.aux,
                                                                 (uint32_t)words, kb, pitch, (uint4*)out);
    else
        dequant_mxfp4_kernel<uint64_t><<<grid, kThreads, 0, s>>>((const uint32_t*)w.packed, (const uint8_t*)w.aux,
                                                                 (uint64_t)words, kb, pitch, (uint4*)out);
    return check_launch("dequant_mxfp4");
}

}  // namespace wq
