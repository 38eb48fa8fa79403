/*
 * tq.h -- C ABI of libtq: TurboQuant-style KV-cache compression on NVIDIA B200 (sm_100a).
 *
 * The hot path, and the page that defines each step:
 *   - key encode:   norm separation, seeded Haar rotation, nearest Lloyd-Max level, bit packing
 *                   ("KV Cache API", compressors.py MSECompressor.compress; "aitherkvcache",
 *                   TurboQuant.encode returning uint8 codes plus f32 norms);
 *   - value encode: grouped affine min/max quantization with fp16 scale and zero
 *                   ("KV Cache API", values.py quantize_values);
 *   - decode:       unpack, codebook gather, inverse rotation, norm rescale; affine dequant for values
 *                   (compressors.py MSECompressor.decompress; values.py dequantize_values);
 *   - decode-step attention scored directly against the packed keys
 *                   ("KV Cache API", store.py TurboQuantKVCache.attention_scores / attend;
 *                   "turbo-attn", the split-K paged decode kernel with a fused query rotation).
 *
 * Conventions shared by every entry point
 *   - Every call returns a tq_status.  On anything but TQ_OK, tq_last_error() returns a message (owned by
 *     the library, valid until the next call on the same thread) that names the offending argument.
 *   - Device pointers are caller-owned (allocate them with any allocator, e.g. PyTorch).  No entry point
 *     allocates or frees device memory except tq_codec_create / tq_codec_destroy.
 *   - Kernels are enqueued on the caller's stream (a cudaStream_t passed as void*; NULL = the legacy
 *     default stream) and return without synchronising.  Outputs are fully overwritten.
 *   - Argument errors are detected on the host before anything is enqueued; nothing is launched then.
 *   - Preconditions that are NOT checked on the device: inputs are finite (no NaN/Inf), pointers
 *     reference allocations of the stated sizes, and outputs do not overlap inputs.
 *   - Half-precision data are IEEE binary16 passed as void* / uint16_t*.
 *   - Supported head dims for the device kernels: 64, 128, 256.  Key bits 1..4.  Value bits 2, 3, 4, 8
 *     with group 32 or group == head_dim (the page's "token" scale layout).
 *   - Packed rows are LSB-first bitstreams: index j of a row occupies bits [j*b, (j+1)*b) of the row read
 *     as little-endian bytes; a row has (d*b + 7) / 8 bytes and rows are contiguous.
 */
#ifndef TQ_H
#define TQ_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum tq_status {
    TQ_OK = 0,
    TQ_ERR_INVALID_ARG = 1,   /* null pointer, negative count, misaligned pointer or stride, bad layout */
    TQ_ERR_UNSUPPORTED = 2,   /* a head_dim / bits / group / GQA combination the kernels do not implement */
    TQ_ERR_CUDA = 3,          /* a CUDA runtime call failed; the message carries cudaGetErrorString */
    TQ_ERR_DEVICE_FLAG = 4    /* a kernel's bounded wait expired and it raised the device error flag */
} tq_status;

typedef enum tq_dtype {
    TQ_F16 = 0,               /* IEEE binary16 */
    TQ_F32 = 1,               /* IEEE binary32 */
    TQ_BF16 = 2               /* bfloat16 (the paged-cache entry points) */
} tq_dtype;

/* Message for the last non-TQ_OK status returned on this thread ("" if none). */
const char* tq_last_error(void);

/* ABI version of this header (major * 100 + minor). */
int tq_version(void);

/* --------------------------------------------------------------------------------------------------
 * Host parameter builders (CPU only; no device needed).
 * ------------------------------------------------------------------------------------------------ */

/*
 * tq_make_rotation -- the seeded Haar rotation Pi ("KV Cache API", compressors.py MSECompressor.__init__:
 * G = randn(d, d); Q, R = qr(G); Pi = Q * sign(diag R), zero signs taken as +1; "TurboQuant: A KV Cache
 * Compression Technique", step 1, Haar-distributed orthogonal matrix).
 *   d        head dimension, 2..1024.
 *   seed     G[i][j] is standard normal draw i*d + j of SplitMix64(seed) through Box-Muller (pairs of
 *            consecutive outputs u1, u2: r = sqrt(-2 ln u1'), draws r cos(2 pi u2'), r sin(2 pi u2'), with
 *            u1' = (u1 >> 11 + 0.5) 2^-53 and u2' = (u2 >> 11) 2^-53).
 *   pi       out, nullable: d*d doubles, row-major; the rotated vector is y = Pi x.
 *   pi_f16   out, nullable: d*d binary16, the nearest fp16 of each entry (Pi_op, what the kernels use).
 * Errors: TQ_ERR_INVALID_ARG for d out of range or both outputs NULL.
 */
tq_status tq_make_rotation(int d, uint64_t seed, double* pi, uint16_t* pi_f16);

/* Rotation kinds of tq_make_rotation_ex / tq_codec_create_ex. */
typedef enum tq_rotation {
    TQ_ROT_HAAR = 0,          /* the seeded Haar rotation of tq_make_rotation */
    TQ_ROT_HADAMARD = 1       /* the seeded randomized Walsh-Hadamard rotation below */
} tq_rotation;

/*
 * tq_make_rotation_ex -- tq_make_rotation for either rotation kind.  TQ_ROT_HADAMARD ("turbo-attn", The
 * codec, "Hadamard rotation": a Walsh-Hadamard transform spreads outlier channels across the vector and the
 * queries are rotated the same way) is Pi = H diag(s) / sqrt(d): H the Sylvester Hadamard matrix
 * (H[i][j] = (-1)^popcount(i & j)), s_j = -1 if the top bit of SplitMix64(seed) output j (0-based) is set,
 * else +1.  The page fixes neither the signs nor the scale; these make Pi orthogonal and the rotated
 * coordinates of an isotropic vector follow the same marginal, so the same codebook applies.
 *   rotation  TQ_ROT_HAAR or TQ_ROT_HADAMARD (then d must be a power of two).
 * Errors: TQ_ERR_INVALID_ARG for a bad kind, d out of range or not a power of two (Hadamard), or both
 * outputs NULL.
 */
tq_status tq_make_rotation_ex(int d, uint64_t seed, int rotation, double* pi, uint16_t* pi_f16);

/*
 * tq_build_codebook -- data-independent Lloyd-Max levels for one rotated coordinate ("KV Cache API",
 * compressors.py calls _solve_codebook(head_dim, bits), body not shown; "TurboQuant: A KV Cache
 * Compression Technique", step 2, optimal codebooks from a mathematical derivation).  The coordinate
 * density is the exact marginal of a uniform point on the unit sphere S^(d-1):
 * f(x) proportional to (1 - x^2)^((d-3)/2) on [-1, 1].
 *   d, bits       2 <= d <= 65536, 1 <= bits <= 8.
 *   centroids     out, nullable: 2^bits doubles, ascending (c*).
 *   centroids_f16 out, nullable: 2^bits binary16, the nearest fp16 of each level (c_op).
 *   boundaries    out, nullable: 2^bits - 1 floats, midpoints of adjacent c_op levels (exact in fp32).
 *   distortion    out, nullable: D = E ||y - Q(y)||^2 for a uniform unit vector y quantized coordinate-wise
 *                 with c_op and these boundaries.
 * Errors: TQ_ERR_INVALID_ARG for d or bits out of range.
 */
tq_status tq_build_codebook(int d, int bits, double* centroids, uint16_t* centroids_f16,
                            float* boundaries, double* distortion);

/* --------------------------------------------------------------------------------------------------
 * Key codec handle: Pi_op, Pi_op^T, c_op, boundaries and search tables resident on the current device.
 * ------------------------------------------------------------------------------------------------ */

typedef struct tq_codec tq_codec;

/*
 * tq_codec_create -- build the rotation and codebook for (d, k_bits, seed) on the host and upload them to
 * the current CUDA device (synchronously, with cudaMalloc/cudaMemcpy; not a hot-path call).
 *   d      64, 128 or 256.       k_bits 1..4.
 *   out    receives the handle; the handle belongs to the device that was current at creation.
 * Errors: TQ_ERR_UNSUPPORTED for other d / bits, TQ_ERR_CUDA if the device allocation fails.
 */
tq_status tq_codec_create(int d, int k_bits, uint64_t seed, tq_codec** out);

/*
 * tq_codec_create_ex -- tq_codec_create with the rotation kind (tq_rotation).  Every kernel is the same:
 * the rotation is a d x d fp16 matrix multiplied on the tensor cores whichever kind it is.
 * Errors: as tq_codec_create, plus TQ_ERR_INVALID_ARG for an unknown kind.
 */
tq_status tq_codec_create_ex(int d, int k_bits, uint64_t seed, int rotation, tq_codec** out);

/* The rotation kind a codec was created with (TQ_ROT_HAAR for tq_codec_create). */
tq_status tq_codec_rotation(const tq_codec* codec, int* rotation);

/* Free a codec (NULL is accepted).  The caller must ensure no enqueued work still uses it. */
tq_status tq_codec_destroy(tq_codec* codec);

/* Read back a codec's parameters (any out pointer may be NULL). */
tq_status tq_codec_info(const tq_codec* codec, int* d, int* k_bits, uint64_t* seed);

/*
 * tq_encode_k -- key encode ("KV Cache API", compressors.py MSECompressor.compress: norms, normalise,
 * rotate, nearest centroid, pack; "aitherkvcache": fp16 [..., 128] -> uint8 [..., 64] at 4 bits + f32 norms).
 *   x             in, device, binary16 rows: row r starts at x + r * x_row_stride (elements).  x must be
 *                 16-byte aligned and x_row_stride a multiple of 8 with x_row_stride >= d.
 *   n             number of rows (0 is a no-op).
 *   slot_mapping  in, device, nullable, int64[n]: destination row of each input row in the output arrays
 *                 (a paged pool); a negative entry skips the row.  NULL: row r goes to row r.
 *   packed        out, device: rows of d*k_bits/8 bytes.      norms  out, device: float per row.
 * Per row: n = ||x||_2 (fp32); y = Pi_op x / (n + 1e-8); index j = #{i : t_i < y_j}; LSB-first packing.
 * Indices agree with the fp64 definition except where y_j lies within ~1e-6 of a boundary t_i.
 */
tq_status tq_encode_k(const tq_codec* codec, const void* x, int64_t n, int64_t x_row_stride,
                      const int64_t* slot_mapping, uint8_t* packed, float* norms, void* stream);

/*
 * tq_decode_k -- key decode ("KV Cache API", compressors.py MSECompressor.decompress: centroids[idx] @ Pi,
 * times the norm).
 *   packed, norms in, device: n rows as written by tq_encode_k (contiguous).
 *   out           out, device: n rows of d elements of out_dtype (TQ_F16 or TQ_F32), 16-byte aligned.
 * x_hat = n * Pi_op^T c_op[idx], accumulated in fp32 on the tensor cores.
 */
tq_status tq_decode_k(const tq_codec* codec, const uint8_t* packed, const float* norms, int64_t n,
                      void* out, int out_dtype, void* stream);

/* --------------------------------------------------------------------------------------------------
 * Value codec (no handle: the format is fully described by d, bits and group).
 * ------------------------------------------------------------------------------------------------ */

/*
 * tq_encode_v -- grouped affine value quantizer ("KV Cache API", values.py quantize_values).
 *   d, bits, group  d in {64,128,256}; bits in {2,3,4,8}; group 32 or d (the page's "token" layout).
 *   x               in, device, binary16 rows with stride x_row_stride (elements; 16-byte aligned rows).
 *   slot_mapping    as for tq_encode_k.
 *   data            out, device: rows of (d*bits+7)/8 bytes.
 *   scales, zeros   out, device: binary16 [rows][d/group].
 * Per group, in IEEE fp32 with one rounding per operation and in this order:
 *   scale = max((max - min) / (2^bits - 1), 1e-12); zero = min;
 *   q = clamp(round_half_even((x - zero) / scale), 0, 2^bits - 1);
 * scale and zero are then stored as fp16 (round to nearest even).  The result is bit-exact with that
 * definition.
 */
tq_status tq_encode_v(int d, int bits, int group, const void* x, int64_t n, int64_t x_row_stride,
                      const int64_t* slot_mapping, uint8_t* data, void* scales, void* zeros, void* stream);

/*
 * tq_decode_v -- value dequantization ("KV Cache API", values.py dequantize_values):
 * x_hat = float(q) * float(scale16) + float(zero16), two fp32 operations, then stored as out_dtype
 * (TQ_F32 exact; TQ_F16 round to nearest even).  Inputs are contiguous rows as tq_encode_v writes them.
 */
tq_status tq_decode_v(int d, int bits, int group, const uint8_t* data, const void* scales,
                      const void* zeros, int64_t n, void* out, int out_dtype, void* stream);

/* --------------------------------------------------------------------------------------------------
 * Decode-step attention over the compressed cache.
 * ------------------------------------------------------------------------------------------------ */

/*
 * Cache layouts.  Every pool array (K payload, K norms, V data, V scales, V zeros) is indexed by a row:
 *   contiguous: row = (b * num_kv_heads + h) * max_seq_len + t;
 *   paged:      row = (block_table[b * max_blocks + t / block_size] * num_kv_heads + h) * block_size
 *                     + t % block_size.
 * Sequence b attends to tokens 0 .. seq_lens[b]-1 (all max_seq_len tokens if seq_lens is NULL in the
 * contiguous layout; seq_lens is required for the paged layout).  The kernels clamp seq_lens[b] to
 * [0, max_seq_len] in the contiguous layout and to [0, max_blocks * block_size] in the paged one, so a length
 * past the cache attends to the whole addressable sequence and never reads beyond its rows or its
 * block-table row.  A negative block_table entry names no block: its tokens are left out (of the
 * softmax; their scores are -inf).  Every other entry below the (clamped) length must name a block of the pools.  Rows of a
 * pool behind a sequence's last token may hold anything; a pool holds one block at least.  Query head hq reads kv head
 * hq / (num_q_heads / num_kv_heads).
 */
typedef struct tq_attend_args {
    int batch;                 /* B, 1 .. 65535 */
    int num_q_heads;           /* H_q, a multiple of num_kv_heads; H_q / H_kv <= 8 */
    int num_kv_heads;          /* H_kv, 1 .. 65535 */
    int head_dim;              /* must equal the codec's d */
    int v_bits;                /* 2, 3, 4 or 8 */
    int v_group;               /* 32 or head_dim */
    float scale;               /* softmax scale; 0 means 1/sqrt(head_dim) ("KV Cache API", attention_scores) */
    int64_t max_seq_len;       /* contiguous layout: T per (b, h); paged: ignored */
    const int32_t* block_table;/* NULL: contiguous layout.  Else device int32 [batch][max_blocks] */
    int max_blocks;            /* paged: columns of block_table */
    int block_size;            /* paged: tokens per block (16) */
    const int32_t* seq_lens;   /* device int32 [batch], nullable in the contiguous layout */
    const void* q;             /* device binary16 [batch][num_q_heads][head_dim] */
    const uint8_t* k_packed;   /* device pool of key rows (tq_encode_k format) */
    const float* k_norms;      /* device pool of key norms */
    const uint8_t* v_data;     /* device pool of value rows (tq_encode_v format) */
    const void* v_scales;      /* device binary16 pool [rows][head_dim / v_group] */
    const void* v_zeros;       /* device binary16 pool [rows][head_dim / v_group] */
    float* out;                /* device float [batch][num_q_heads][head_dim] */
    void* workspace;           /* device scratch (16-byte aligned) of at least the size
                                  tq_attend_workspace_bytes reports: the prepared query fragments of each
                                  (sequence, kv head), then the split-K partials.  Its contents need no
                                  initialisation and are overwritten by every call. */
    size_t workspace_bytes;
} tq_attend_args;

/*
 * tq_attend_workspace_bytes -- bytes of workspace tq_attend_decode needs for these arguments on the current
 * device: (head_dim / 16 * 32 + 2) * 16 bytes per (sequence, kv head) for the prepared query, plus the split-K
 * partials when the sequence axis is split.  Only the shape fields of args are read.  The size assumes the
 * most splits any key width can use (four attention CTAs per SM); a launch whose kernel keeps fewer CTAs
 * resident splits less and uses a prefix of the same workspace.
 * Errors: the same argument checks as tq_attend_decode (TQ_ERR_INVALID_ARG / TQ_ERR_UNSUPPORTED).
 */
tq_status tq_attend_workspace_bytes(const tq_attend_args* args, size_t* bytes);

/*
 * tq_attend_decode -- one decode step of attention against the compressed cache ("KV Cache API",
 * store.py attention_scores + softmax + attend; "turbo-attn", split-K paged decode with the query
 * rotated once).  For each (b, hq) with h = hq / G:
 *   q_rot = Pi_op q;  s_t = scale * n_t * <q_rot, c_op[idx_t]>;  p = softmax(s);
 *   out = sum_t p_t * (q_t * scale16_t + zero16_t)   (the value dequantized inside the kernel).
 * No fp16 key or value is written to memory.  A sequence of length 0 yields zeros.  A small first kernel
 * rotates and splits the query once per (sequence, kv head); the attention kernel is its programmatic
 * dependent on the same stream.  When the sequence axis is split over several CTAs, a third kernel (again a
 * programmatic dependent) merges the per-split partials with a log-sum-exp rescale.  Calls that overlap on
 * the GPU must use distinct workspaces.
 */
tq_status tq_attend_decode(const tq_codec* codec, const tq_attend_args* args, void* stream);

/*
 * tq_attend_scores -- the attention logits of the compressed path, for score-fidelity measurements
 * ("turboquant-pytorch", V3: Attention Score Accuracy -- cosine similarity and top-1 / top-5 matches of the
 * scores against the uncompressed ones): s[b][hq][t] = scale * n_t * <Pi_op q, c_op[idx_t]> in fp32, the
 * same scores tq_attend_decode softmaxes.
 *   scores  out, device float [batch][num_q_heads][L], L = max_seq_len (contiguous) or max_blocks * 16
 *           (paged); positions at or past a sequence's length are -inf.
 * args->out and the value pool are not used; args->workspace needs at least tq_attend_workspace_bytes bytes
 * (only its prepared-query part is written).
 * Errors: as tq_attend_decode.
 */
tq_status tq_attend_scores(const tq_codec* codec, const tq_attend_args* args, float* scores, void* stream);

/* --------------------------------------------------------------------------------------------------
 * Attention with a window of recent uncompressed tokens.
 * ------------------------------------------------------------------------------------------------ */

/* Largest window per (sequence, kv head) tq_attend_decode_window accepts. */
#define TQ_ATTEND_WINDOW_MAX 256

typedef struct tq_attend_window {
    const void* k;             /* device binary16 [batch][num_kv_heads][max_len][head_dim]: recent keys as stored */
    const void* v;             /* device binary16, same layout: recent values as stored */
    const int32_t* lens;       /* device int32 [batch]: window tokens of each sequence (clamped to 0..max_len);
                                  NULL: max_len for every sequence */
    int max_len;               /* 1..TQ_ATTEND_WINDOW_MAX */
} tq_attend_window;

/*
 * tq_attend_window_workspace_bytes -- workspace bytes tq_attend_decode_window needs (as
 * tq_attend_workspace_bytes, with one more partial per (sequence, kv head) for the window).
 */
tq_status tq_attend_window_workspace_bytes(const tq_attend_args* args, const tq_attend_window* window,
                                           size_t* bytes);

/*
 * tq_attend_decode_window -- tq_attend_decode over the compressed cache plus a window of recent tokens kept
 * uncompressed ("KV Cache API", store.py TurboQuantKVCache: attention_scores concatenates the quantized
 * part's scores with scale * query @ key_buffer^T; the softmax runs over both; attend adds the quantized
 * part's weights times the dequantized values and the buffer's weights times the buffer's values).  The
 * window's scores are fp32 dot products of the fp16 query and keys, times the same scale; one extra CTA per
 * (sequence, kv head) computes them and its partial (max, sum, weighted values) enters the same split merge.
 * A sequence whose compressed part and window are both empty yields zeros.
 * Errors: as tq_attend_decode, plus TQ_ERR_INVALID_ARG for a NULL window, NULL k or v, max_len outside
 * 1..TQ_ATTEND_WINDOW_MAX or misaligned (16-byte) k / v.
 */
tq_status tq_attend_decode_window(const tq_codec* codec, const tq_attend_args* args, const tq_attend_window* window,
                                  void* stream);

/*
 * TQ_ATTEND_SCRATCH_BYTES -- size of the library-owned scratch used by tq_attend_decode_noalloc (4 MiB).
 * That array lives in the library's device image, so every GPU that loads libtq holds it until the process
 * exits, whether or not the entry point is ever called.
 */
#define TQ_ATTEND_SCRATCH_BYTES (4u << 20)

/*
 * tq_attend_decode_noalloc -- the same decode-step attention as tq_attend_decode, for callers that cannot
 * allocate device memory at all: code running inside a CUDA graph that is being captured or replayed, a
 * serving loop whose memory pool is fixed once at start-up, or a host process that only receives a
 * stream and buffers from elsewhere.  The pages have no counterpart; this is a property of this library.
 *
 * Instead of a caller workspace it uses a fixed scratch array of TQ_ATTEND_SCRATCH_BYTES that the library
 * declares at file scope in device memory; args->workspace and args->workspace_bytes are ignored.  The
 * entry point calls no allocator (no cudaMalloc, no cudaFree, nothing that allocates).
 *   - Set-up: the first call on each device looks up the scratch array's device address with
 *     cudaGetSymbolAddress (with that device current) and caches it for the life of the process; make that
 *     first call outside any stream capture.  The cached address belongs to the device's primary context:
 *     after cudaDeviceReset (or any reset of that context) it is stale, so do not call this entry point
 *     again in a process that has reset the device.
 *   - Limit: the check uses the size tq_attend_workspace_bytes reports for the same arguments (planned for
 *     the most splits any key width can use); when that exceeds TQ_ATTEND_SCRATCH_BYTES the call is
 *     rejected with TQ_ERR_INVALID_ARG and a message giving both sizes, even if this codec's key width
 *     would launch fewer splits.  Use tq_attend_decode with a caller workspace for such shapes.
 *   - Sharing: all calls on a device share the one array and it keeps the last call's contents; nothing
 *     in it needs to start at zero, since every launch overwrites the part it reads.  Calls that can
 *     overlap on the GPU (different streams without ordering, or different threads) race on it and must
 *     be serialised by the caller.
 * Errors: as tq_attend_decode, plus TQ_ERR_CUDA if the address lookup fails.
 */
tq_status tq_attend_decode_noalloc(const tq_codec* codec, const tq_attend_args* args, void* stream);

/* --------------------------------------------------------------------------------------------------
 * QJL residual keys.
 * ------------------------------------------------------------------------------------------------ */

/*
 * tq_codec_create_qjl -- a key codec for QJL residual keys ("KV Cache API", compressors.py
 * TurboQuantCompressorV2: the MSE compressor at bits - 1, then one sign bit per row of a seeded Gaussian matrix S
 * applied to the residual r of the MSE reconstruction, and ||r||).
 *   bits      total bits per coordinate, 2..5; the MSE stage uses bits - 1 (tq_codec_info reports bits - 1, so
 *             the codec also serves tq_encode_k / tq_decode_k / tq_attend_decode as an ordinary key codec).
 *   S         d x d, entry (i, j) = Gaussian draw i * d + j of this library's generator (SplitMix64 and
 *             Box-Muller) seeded with seed + 10000; the tensor cores multiply by S_op = fp16(S).
 * Errors: as tq_codec_create_ex, TQ_ERR_UNSUPPORTED for bits outside 2..5.
 */
tq_status tq_codec_create_qjl(int d, int bits, uint64_t seed, int rotation, tq_codec** out);

/*
 * tq_make_qjl_matrix -- the sketch S of a QJL codec with this d and seed, on the host (row-major d*d): entry
 * (i, j) is Gaussian draw i * d + j of the generator seeded with seed + 10000; s_f16 (nullable) receives
 * fp16(S), the operand the kernels use.  Either output may be NULL, not both.
 */
tq_status tq_make_qjl_matrix(int d, uint64_t seed, double* s, uint16_t* s_f16);

/* tq_codec_qjl_bits -- the total bits of a QJL codec; 0 for a codec made by tq_codec_create / _ex. */
tq_status tq_codec_qjl_bits(const tq_codec* codec, int* bits);

/*
 * tq_encode_k_qjl -- QJL key encode ("KV Cache API", compressors.py TurboQuantCompressorV2.compress):
 *   the MSE stage, exactly tq_encode_k with this codec at bits - 1, into packed and norms; then
 *   k_mse = n * Pi_op^T c_op[idx];  r = x - k_mse (f32);  rho = ||r|| (f32);  sign_i = ((S_op r)_i >= 0).
 *   signs     out, device: rows of d/8 bytes; coordinate i is bit i of the row's LSB-first bitstream, 1 for +1.
 *   rho       out, device: float per row.
 * Rows, strides, alignment and the slot mapping (which places packed, norms, signs and rho alike) are those of
 * tq_encode_k.  k_mse multiplies fp16 codebook values by fp16 Pi_op and S_op r multiplies r, split into fp16
 * hi + lo halves, by fp16 S_op, both with f32 accumulation: a sign can differ from an exact evaluation only
 * where (S_op r)_i lies within about 1e-6 * ||S_op row i|| * ||x|| of zero.  Launches two kernels on `stream`.
 * Errors: as tq_encode_k; TQ_ERR_INVALID_ARG for a codec not made by tq_codec_create_qjl or NULL signs / rho.
 */
tq_status tq_encode_k_qjl(const tq_codec* codec, const void* x, int64_t n, int64_t x_row_stride,
                          const int64_t* slot_mapping, uint8_t* packed, float* norms, uint8_t* signs, float* rho,
                          void* stream);

/* QJL key pools beside the MSE-stage pools of tq_attend_args, indexed by the same rows. */
typedef struct tq_qjl_keys {
    const uint8_t* signs;      /* device pool of sign rows (tq_encode_k_qjl format: d/8 bytes per row) */
    const float* rho;          /* device pool of residual norms */
} tq_qjl_keys;

/*
 * tq_attend_qjl_workspace_bytes -- workspace bytes tq_attend_decode_qjl needs: as tq_attend_workspace_bytes, with
 * a second block of prepared query fragments (the sketched query) per (sequence, kv head).
 */
tq_status tq_attend_qjl_workspace_bytes(const tq_attend_args* args, size_t* bytes);

/*
 * tq_attend_decode_qjl -- decode attention over QJL residual keys ("KV Cache API", store.py attention_scores
 * with compressors.py asymmetric_attention_scores): for each (b, hq), kv head h = hq / G,
 *   s_t = scale * ( n_t <Pi_op q, c_op[idx_t]> + rho_t sqrt(pi/2) / d <S_op q, sign_t> ),  sign_t in {-1, +1}^d,
 *   p = softmax(s);  out = sum_t p_t * (q_t * scale16_t + zero16_t),
 * i.e. tq_attend_decode with the estimator's second term in every logit.  args describes the MSE-stage pools
 * (the codec's bits - 1 codes and norms) and the values exactly as for tq_attend_decode; keys adds the sign and
 * rho pools.  The prepared query now has two halves (Pi_op q and S_op q, each fp16 hi + lo fragments); the sign
 * pairs enter the tensor cores as fp16 +-1.  Values: 2 or 4 bits in groups of 32.
 * Errors: as tq_attend_decode; TQ_ERR_INVALID_ARG for a codec not made by tq_codec_create_qjl, NULL or
 * misaligned (16-byte) signs / rho; TQ_ERR_UNSUPPORTED for another value format.
 */
tq_status tq_attend_decode_qjl(const tq_codec* codec, const tq_attend_args* args, const tq_qjl_keys* keys,
                               void* stream);

/* --------------------------------------------------------------------------------------------------
 * The paged cache: block tables and slots, uncompressed pages, page selection.
 *
 * A page is one block of 16 tokens of the paged layout above.  Head page e = page * num_kv_heads + h is the 16 rows
 * of kv head h in a page; a slot e * 16 + t % 16 is the pool row of one token and kv head, for compressed pools
 * (tq_encode_k, tq_encode_v) and uncompressed ones alike.  An uncompressed pool is
 * [num_pages][num_kv_heads][16][head_dim] of binary16 or bfloat16.
 *
 * One decode step over a paged cache: tq_plan_pages gives every request's new tokens their pages and slots;
 * tq_encode_k / tq_encode_v, or tq_append_pages for layers kept uncompressed, store them; tq_attend_decode or
 * tq_attend_pages read the cache.  To read only part of a long cache, tq_append_pages keeps channel bounds of every
 * page's keys, tq_select_pages picks pages by them, and either attention reads the picked ones.
 *
 * No call synchronises, allocates, or keeps anything between calls, so each can be captured into a CUDA graph and
 * replayed with new contents of the same buffers.  Page ids that name no page of a pool are never followed by the calls
 * below: their tokens are left out.  tq_attend_decode, which is not told how many blocks its pools hold, leaves out
 * negative ids only.
 * ------------------------------------------------------------------------------------------------ */

typedef struct tq_plan_args {
    int batch;                 /* requests, 1 .. 2^24 */
    int num_kv_heads;          /* 1 .. 1024 */
    int max_blocks;            /* columns of block_table */
    int num_pages;             /* pages of the pool; entries of free_pages */
    int64_t max_tokens;        /* input rows (tokens) the caller has: slots for this many are written */
    const int32_t* new_lens;   /* device [batch]: tokens to add; 0 none; negative: the request is finished */
    const int32_t* seq_lens;   /* device [batch]: tokens cached so far (clamped to 0 .. max_blocks * 16) */
    int32_t* block_table;      /* device [batch][max_blocks], updated in place: entries of new pages are written */
    int32_t* free_pages;       /* device [num_pages], updated in place: a ring of free page ids */
    const int32_t* free_state; /* device [2]: index of the ring's first free page, number of free pages */
    int64_t* slots;            /* out, device [max_tokens][num_kv_heads] (may be NULL if max_tokens is 0) */
    int32_t* row_start;        /* out, device [batch + 1]: first input row of each request; the last entry is their sum */
    int32_t* start_pos;        /* out, device [batch]: position of a request's first new token, -1 if it adds none
                                  because it was refused or is finished */
    int32_t* seq_lens_out;     /* out, device [batch]: tokens after this step (may be seq_lens) */
    int32_t* free_state_out;   /* out, device [2] (may be free_state) */
} tq_plan_args;

/*
 * tq_plan_pages -- block tables and slots of one step, from the requests' lengths, on the GPU.  The input rows of
 * request b are row_start[b] .. row_start[b + 1] - 1 (row_start: running sum of max(new_lens, 0)); its i-th new token
 * is token seq_lens[b] + i and gets
 *   slots[(row_start[b] + i) * num_kv_heads + h] = (block_table[b][t / 16] * num_kv_heads + h) * 16 + t % 16.
 *   - Pages: a request needs ceil((len + new) / 16) - ceil(len / 16) pages.  In the order of the batch, it is refused
 *     if its tokens do not fit its table row or max_tokens, or if it needs pages and the needs up to and including
 *     it exceed the free count (so no later request that needs pages gets any either).  A refused request adds
 *     nothing; its length and table row stay as they are.
 *   - New pages come from the ring's start in the order of the batch.  A finished request's pages (the
 *     ceil(len / 16) entries of its table row) are put at the ring's end, for later calls, and its length becomes 0.
 *   - Rows of refused requests, rows from row_start[batch] on, and rows whose table entry names no page get slot -1,
 *     which tq_encode_k, tq_encode_v and tq_append_pages skip.
 * Preconditions not checked: a page id is owned once (in one table row or in the ring), seq_lens are those of the table
 * rows, and no output overlaps an input but for the two pairs named above.  row_start saturates at 2^31 - 1 (requests from there on are refused).
 * Errors: TQ_ERR_INVALID_ARG for counts out of range, NULL or misaligned pointers.
 */
tq_status tq_plan_pages(const tq_plan_args* args, void* stream);

typedef struct tq_append_args {
    int dtype;                 /* TQ_F16 or TQ_BF16: k, v, pools and bounds */
    int head_dim;              /* 64, 128 or 256 */
    int num_kv_heads;
    int num_pages;             /* pages of the pools and of bounds */
    int64_t num_tokens;        /* input rows (0 is a no-op) */
    const void* k;             /* device: token t, kv head h at k + t * k_token_stride + h * k_head_stride (elements) */
    const void* v;             /* device, the same with its own strides; needed if v_pool is given */
    int64_t k_token_stride, k_head_stride, v_token_stride, v_head_stride;   /* multiples of 8 */
    const int64_t* slots;      /* device [num_tokens][num_kv_heads], e.g. from tq_plan_pages; slots below 0 or past the
                                  pool's rows skip the row */
    void* k_pool;              /* nullable: device [num_pages][num_kv_heads][16][head_dim] */
    void* v_pool;              /* nullable, the same shape */
    void* bounds;              /* nullable: device [num_pages][num_kv_heads][2][head_dim]: lowest, highest key */
} tq_append_args;

/*
 * tq_append_pages -- store new keys and values of a step in uncompressed pools, and keep the channel bounds of the
 * pages' keys: bounds[page][h][0][c] and [1][c] are the minimum and maximum over the page's keys of channel c.  A
 * page whose first token (slot % 16 == 0) is among the rows starts anew; others extend the bounds they have.  For a
 * compressed cache only bounds is given and the rows go through tq_encode_k.
 * A key that is not a number counts in its page's bounds only if the channel has no other.  Rows not named by a slot are
 * left as they were.  Tokens of one page and kv head must be consecutive input rows, as
 * tq_plan_pages lays them out (a page that appears in two places in one call gets undefined bounds); if a slot appears
 * twice, one of its rows is stored.
 * Errors: TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED (head_dim, dtype).
 */
tq_status tq_append_pages(const tq_append_args* args, void* stream);

typedef struct tq_select_args {
    int dtype;                 /* TQ_F16 or TQ_BF16: q and bounds */
    int batch, num_q_heads, num_kv_heads, head_dim;
    int max_blocks;            /* columns of block_table */
    int num_pages;             /* pages of bounds */
    int budget;                /* pages kept per (sequence, kv head) */
    int keep_first, keep_last; /* pages at the start and at the end that are kept whatever their score
                                  (keep_first >= 0, keep_last >= 1, keep_first + keep_last <= budget) */
    const void* q;             /* device [batch] rows of [num_q_heads][head_dim], q_stride elements apart */
    int64_t q_stride;          /* a multiple of 8 */
    const void* bounds;        /* device [num_pages][num_kv_heads][2][head_dim] (tq_append_pages) */
    const int32_t* block_table;/* device [batch][max_blocks] */
    const int32_t* seq_lens;   /* device [batch] (clamped to 0 .. max_blocks * 16) */
    int32_t* pages;            /* out, device [batch][num_kv_heads][budget]: head pages in ascending order, then -1 */
    int32_t* lens;             /* out, device [batch][num_kv_heads]: tokens of the listed pages */
    void* workspace;           /* device scratch (16-byte aligned; may be NULL if none is needed): the scores of a call
                                  with few rows; needs no initialisation, overwritten by every call that uses it */
    size_t workspace_bytes;
} tq_select_args;

/*
 * tq_select_pages_workspace_bytes -- bytes of workspace tq_select_pages needs for these shapes on the current device:
 * 0, or about 4 * batch * num_kv_heads * max_blocks when there are fewer (sequence, kv head) rows than SMs or rows are very
 * long.  Only the shape fields are read.
 */
tq_status tq_select_pages_workspace_bytes(const tq_select_args* args, size_t* bytes);

/*
 * tq_select_pages -- the pages a decode step attends to.  For each page of a sequence and each kv head,
 *   score = max over the group's query heads of  sum_c max(q_c * bounds[0][c], q_c * bounds[1][c]),
 * an upper bound of q . k over the page's keys.  The first keep_first and last keep_last pages are kept; the rest of
 * `budget` goes to the highest scores, ties to the lower index.  A sequence of at most `budget` pages keeps all.
 * lens counts the tokens of the listed pages (every page is full but a sequence's last, which is always listed last),
 * so pages and lens are a block table and lengths with one row per (sequence, kv head).  Read them with
 * tq_attend_pages (selected = 1), or with tq_attend_decode on the compressed pools as batch * num_kv_heads sequences
 * of one kv head (at most 65535 of them): a head page is a page of a pool with one kv head.  A listed page whose table entry names no page is
 * given as -1, which either attention leaves out.
 * Sums run in fp32 in a fixed order (per 8 channels an even and an odd chain, then halves added to halves), so the
 * result is the same on every run and for every shape of the call.  A score that is not a number ranks last; a NaN in
 * the query counts as 0.  An infinite bound counts as the formula has it (0 times infinity is not a number).  The bounds are
 * those of tq_append_pages: [0] nowhere above [1].  (Which pages are kept is undefined among those where the finite terms
 * of sum_c |q_c bounds_c| add up to more than 2^126 or less than 2^-100, and for an infinite query.)
 * Calls that overlap on the GPU must use distinct workspaces.
 * Errors: TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED (head_dim, dtype, GQA group > 8, 2^39 pages or more in all rows).
 */
tq_status tq_select_pages(const tq_select_args* args, void* stream);

typedef struct tq_attend_pages_args {
    int dtype;                 /* TQ_F16 or TQ_BF16: q and pools */
    int batch, num_q_heads, num_kv_heads, head_dim;
    int max_blocks;            /* columns of block_table */
    int num_pages;             /* pages of the pools */
    int selected;              /* 0: block_table [batch][max_blocks] of pages, seq_lens [batch];
                                  1: block_table [batch][num_kv_heads][max_blocks] of head pages, seq_lens
                                     [batch][num_kv_heads] (tq_select_pages) */
    float scale;               /* softmax scale; 0 means 1/sqrt(head_dim) */
    const void* q;             /* device [batch] rows of [num_q_heads][head_dim], q_stride elements apart */
    int64_t q_stride;          /* a multiple of 8 */
    const void* k_pool;        /* device: pages of [num_kv_heads][16][head_dim], k_page_stride elements apart */
    const void* v_pool;
    int64_t k_page_stride, v_page_stride;  /* multiples of 8; num_kv_heads * 16 * head_dim when selected is 1 */
    const int32_t* block_table;/* device int32; entries past a row's length are not read */
    const int32_t* seq_lens;   /* device int32 (clamped to 0 .. max_blocks * 16) */
    float* out;                /* device float [batch][num_q_heads][head_dim] */
    void* workspace;           /* device scratch (16-byte aligned; may be NULL if none is needed); needs no
                                  initialisation, overwritten by every call */
    size_t workspace_bytes;
} tq_attend_pages_args;

/*
 * tq_attend_pages_workspace_bytes -- bytes of workspace tq_attend_pages needs for these shapes on the current device
 * (never more than 8 MiB on a B200; 0 for table rows of up to 32 pages).  Only the shape fields are read.
 */
tq_status tq_attend_pages_workspace_bytes(const tq_attend_pages_args* args, size_t* bytes);

/*
 * tq_attend_pages -- attention of one new token per sequence over uncompressed pages: for each (b, hq), h = hq / G,
 *   p = softmax_t(scale * q . k_t),  out = sum_t p_t v_t   over tokens 0 .. seq_lens[b] - 1.
 * Scores, softmax and sums are fp32.  Rows of a page behind the sequence's last token may hold anything.  A sequence
 * of length 0, or whose table entries name no page, yields zeros, and so does one whose every score is -infinity.  A NaN
 * in a token's key or in the query, or a score of +infinity, makes the head's output NaN, an infinity or NaN in a value
 * its column of it.  The cache is read once, in equal shares per CTA
 * whatever the lengths; a second kernel (a programmatic dependent) joins the sequences that lie in several shares.
 * The same inputs give the same bits on every run.  Calls that overlap on the GPU must use distinct workspaces.
 * Errors: TQ_ERR_INVALID_ARG, TQ_ERR_UNSUPPORTED (head_dim, dtype, GQA group > 8).
 */
tq_status tq_attend_pages(const tq_attend_pages_args* args, void* stream);

/* --------------------------------------------------------------------------------------------------
 * Diagnostics.
 * ------------------------------------------------------------------------------------------------ */

/*
 * Read (and optionally clear) the current device's error flag, which a kernel sets when one of its bounded
 * waits expires.  Synchronises the device.  flag_out receives 0 when nothing was raised.
 */
tq_status tq_read_device_flag(int* flag_out, int clear);

/*
 * tq_stream_status -- wait for the work queued on `stream` (that stream only; other streams keep running) and
 * report whether any kernel's bounded wait has expired: TQ_ERR_DEVICE_FLAG (with the flag in tq_last_error)
 * if the device's error flag is set, else TQ_OK.  clear != 0 resets the flag after reading it.  A kernel
 * whose wait expired has stopped its roles, let every copy and tensor-core operation it issued complete,
 * released its tensor memory and returned, so the context stays usable; its outputs are incomplete.
 */
tq_status tq_stream_status(void* stream, int clear);

/*
 * tq_debug_encode_k_stalled -- a test of the bounded-wait path: tq_encode_k on n contiguous rows (row stride d)
 * with the first 128-row tile's copy withheld in every CTA and every wait limited to wait_limit_cycles
 * (1000 .. 2^31).  Nothing waits on a copy or an MMA that was issued and is still in flight: the waits on
 * the withheld tile run out, the kernel raises the device flag, drains what it issued, frees its tensor memory
 * and returns.  Follow with tq_stream_status to read the result.  The outputs are not meaningful.
 */
tq_status tq_debug_encode_k_stalled(const tq_codec* codec, const void* x, int64_t n, uint8_t* packed, float* norms,
                                    long long wait_limit_cycles, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* TQ_H */
