// The 4-bit K/V cache: its layout in device memory and the launch functions of
// the operators on it (kie_kv4.cu).  Plain C++; included by host and device code.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

// One position of one K/V head is D/2 bytes of codes and D/g (scale, zero) fp16
// pairs, K and V apart:
//
//   codes  [batch][head][ctx_pad][D/8] 32-bit words
//   params [batch][head][ctx_pad/8] blocks of 8 positions, 32 D/g bytes each
//
// ctx_pad is max_ctx rounded up to 64 positions, so that every head starts on a
// 256-byte boundary and whole tiles of positions lie inside the head's memory.
//
// Codes and params are stored in the order in which a warp's matrix fragments
// take them, so that one vector load per lane feeds whole m16n8k16 operands:
//   K word t*(D/32) + b holds channels 32b + 8t + n in nibble n (t = 0..3): lane
//     t of a quad reads its D/32 words, one per 32-channel block, in one load;
//   V 16-bit unit g*(D/32) + b holds channels 32b + 4g + n in nibble n (g = 0..7):
//     lane group g reads its units of a position in one load, and two positions'
//     units merge into the pairs of an operand;
//   row 2t + e of an operand's 8 positions is position t of the block (e = 0) or
//     7 - t (e = 1): the pairs (0,7) (1,6) (2,5) (3,4) read the codes without bank
//     conflicts;
//   K block: per position its fp16 scales, then its zeros;
//   V block: per pair t words [group] of the scales, then of the zeros (positions
//     run along the operand there).
struct Kv4 {
    uint8_t *kc, *vc;        // codes
    uint16_t *kp, *vp;       // params, fp16 bits
    int32_t batch, heads, max_ctx, ctx_pad, dim, group;
};

struct Kv4Strides { int64_t b, t, h; };   // elements between requests, tokens, heads (channels are contiguous)

enum Kv4Type { KV4_F16 = 0, KV4_BF16 = 1, KV4_F32 = 2 };

static inline int kv4_pad(int max_ctx) { return (max_ctx + 63) / 64 * 64; }

// Arguments of kie_launch_kv4_attention.
struct Kv4Attn {
    Kv4 c;
    const void* q;
    void* out;
    Kv4Strides qs, os;
    int32_t type;            // Kv4Type of q and out
    int32_t heads;           // query heads, a multiple of c.heads
    int32_t n_q;             // query tokens per request (rows of q)
    const int32_t* kv_len;   // [batch]
    const int32_t* n_tok;    // [batch] or null: n_q
    int32_t causal, window;
    float scale;
    float* ws;               // partial results
};

extern "C" cudaError_t kie_launch_kv4_append(const Kv4* c, const void* k, const void* v, const Kv4Strides* ks,
                                             const Kv4Strides* vs, int type, int n, const int32_t* start,
                                             const int32_t* n_tok, cudaStream_t st);
extern "C" cudaError_t kie_launch_kv4_read(const Kv4* c, void* k, void* v, const Kv4Strides* ks, const Kv4Strides* vs,
                                           int type, int n, const int32_t* start, const int32_t* n_tok,
                                           cudaStream_t st);
// Floats of workspace that the attention needs on a GPU with `sms` SMs (0 for most
// single-token calls); the pointers of `a` are not looked at.
extern "C" size_t kie_kv4_attention_ws_floats(const Kv4Attn* a, int sms);
extern "C" cudaError_t kie_launch_kv4_attention(const Kv4Attn* a, int sms, cudaStream_t st);

// The same for many tokens of bf16 (kie_kv4_chunk.cu), and a model of its time.
extern "C" double kie_kv4_chunk_us(const Kv4Attn* a, int sms);
extern "C" size_t kie_kv4_chunk_ws_floats(const Kv4Attn* a, int sms);
extern "C" cudaError_t kie_launch_kv4_chunk(const Kv4Attn* a, int sms, cudaStream_t st);
