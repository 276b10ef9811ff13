/*
 * A plain C11 client of the rotary positions, the 4-bit cache and its
 * attention: include/gq.h plus the HIP runtime's C interface, no Python.
 * Results with a closed form:
 *
 *   Keys and values of integers -8 .. 7 with a -8 in every block have a block
 *   scale of 1, so the cache holds them exactly and gq_kv4_read returns them.
 *   With a softmax scale of 0 all weights are equal: row t of a causal prompt
 *   is the mean of the values 0 .. t.
 *   At position 0 a rotation changes nothing.
 *
 * Prints "c client ok" and exits 0 on success; any mismatch prints the case
 * and exits 1. Built by __graft_entry__.build(); run by
 * tests/test_gpu_c_client_kv4.py.
 */
#include <hip/hip_runtime_api.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "gq.h"

#define TOK 40
#define HD 64
#define KV 2
#define HEADS 6
#define PAGE 16
#define PAGES 5

static int failures = 0;

static void check(int ok, const char* what) {
    if (!ok) {
        fprintf(stderr, "c client: FAILED %s\n", what);
        fflush(stderr);
        failures++;
    }
}

static void hip(hipError_t e, const char* what) {
    if (e != hipSuccess) {
        fprintf(stderr, "c client: %s: %s\n", what, hipGetErrorString(e));
        exit(2);
    }
}

static void* device(const void* host, size_t bytes) {
    void* p = NULL;
    hip(hipMalloc(&p, bytes), "hipMalloc");
    if (host) hip(hipMemcpy(p, host, bytes, hipMemcpyHostToDevice), "copy to the GPU");
    return p;
}

/* a small deterministic generator (64-bit LCG, top bits) */
static uint64_t state = 0x9E3779B97F4A7C15ull;
static int next_int(int lo, int hi) {
    state = state * 6364136223846793005ull + 1442695040888963407ull;
    return lo + (int)((state >> 33) % (uint64_t)(hi - lo + 1));
}

int main(void) {
    static float k[TOK][KV][HD], v[TOK][KV][HD], q[TOK][HEADS][HD];
    static float K[TOK][KV][HD], V[TOK][KV][HD], out[TOK][HEADS][HD], turned[TOK][HEADS][HD];
    for (int t = 0; t < TOK; ++t) {
        for (int h = 0; h < KV; ++h) {
            for (int c = 0; c < HD; ++c) {
                k[t][h][c] = (float)next_int(-7, 7);
                v[t][h][c] = (float)next_int(-7, 7);
            }
            for (int b = 0; b < HD / 32; ++b) {
                k[t][h][32 * b + next_int(0, 31)] = -8.f;
                v[t][h][32 * b + next_int(0, 31)] = -8.f;
            }
        }
        for (int h = 0; h < HEADS; ++h)
            for (int c = 0; c < HD; ++c) q[t][h][c] = 0.25f * (float)next_int(-9, 9);
    }

    const int64_t page = gq_kv4_page_bytes(PAGE, KV, HD);
    check(page == (int64_t)PAGE * KV * HD * 9 / 8, "gq_kv4_page_bytes");
    check(gq_kv4_page_bytes(24, KV, HD) < 0, "gq_kv4_page_bytes (not a power of two)");
    float freqs[HD / 2], mscale = 0.f;
    check(gq_rope_freqs(HD, 10000.0, GQ_ROPE_PLAIN, 1.0, 0.0, 0.0, 0.0, freqs, &mscale) == GQ_OK, "gq_rope_freqs");
    check(freqs[0] == 1.f && fabsf(freqs[HD / 4] - 0.01f) < 1e-8f && mscale == 1.f, "frequencies");

    const int32_t table[3] = {3, 0, 4}, start[2] = {0, TOK}, len = TOK;
    int32_t zeros[TOK];
    memset(zeros, 0, sizeof zeros);
    gq_kv4 cache = {device(NULL, (size_t)(PAGES * page)), PAGES, PAGE, KV, HD, device(table, sizeof table), 3, 1};
    int32_t* d_start = device(start, sizeof start);
    int32_t* d_len = device(&len, sizeof len);
    int32_t* d_pos = device(zeros, sizeof zeros);
    float *d_k = device(k, sizeof k), *d_v = device(v, sizeof v), *d_q = device(q, sizeof q);
    float *d_K = device(NULL, sizeof K), *d_V = device(NULL, sizeof V), *d_out = device(NULL, sizeof out);

    /* a rotation by nothing, and its refusals */
    const gq_rope rope = {device(freqs, sizeof freqs), HD, 0, 1.f};
    check(gq_qk_rope(d_q, HEADS * HD, TOK, HEADS, HD, d_pos, &rope, NULL, 0.f, d_out, HEADS * HD, NULL) == GQ_OK, "gq_qk_rope");
    hip(hipMemcpy(turned, d_out, sizeof turned, hipMemcpyDeviceToHost), "copy of the queries");
    check(memcmp(turned, q, sizeof q) == 0, "a rotation at position 0");
    check(gq_qk_rope(d_q, HEADS * HD, TOK, HEADS, HD, d_pos, &rope, NULL, 0.f, d_q + 4, HEADS * HD, NULL) == GQ_ERR_OVERLAP,
          "gq_qk_rope onto its input");

    /* append on a stream of its own, read back */
    hipStream_t s;
    hip(hipStreamCreate(&s), "hipStreamCreate");
    check(gq_kv4_append(&cache, d_k, KV * HD, d_v, KV * HD, TOK, d_start, d_len, NULL, NULL, NULL, 0, 0, NULL, NULL, 0, 0.f,
                        s) == GQ_OK, "gq_kv4_append");
    check(gq_kv4_read(&cache, TOK, d_start, d_len, d_K, d_V, s) == GQ_OK, "gq_kv4_read");
    hip(hipStreamSynchronize(s), "hipStreamSynchronize");
    hip(hipMemcpy(K, d_K, sizeof K, hipMemcpyDeviceToHost), "copy of the keys");
    hip(hipMemcpy(V, d_V, sizeof V, hipMemcpyDeviceToHost), "copy of the values");
    check(memcmp(K, k, sizeof k) == 0 && memcmp(V, v, sizeof v) == 0, "the held values");

    /* the prompt with equal weights: means of the values so far */
    const int64_t need = gq_kv4_attn_ws_bytes(&cache, HEADS, TOK, 3 * PAGE);
    check(need >= 0, "gq_kv4_attn_ws_bytes");
    void* ws = need ? device(NULL, (size_t)need) : NULL;
    check(gq_kv4_attn(&cache, d_q, HEADS * HD, HEADS, TOK, d_start, d_len, TOK, 3 * PAGE, 0.f, 1, 0, d_out, HEADS * HD, ws, need,
                      s) == GQ_OK, "gq_kv4_attn");
    hip(hipStreamSynchronize(s), "hipStreamSynchronize");
    hip(hipMemcpy(out, d_out, sizeof out, hipMemcpyDeviceToHost), "copy of the output");
    int bad = 0;
    for (int h = 0; h < HEADS; ++h)
        for (int c = 0; c < HD; ++c) {
            double sum = 0.0;
            for (int t = 0; t < TOK; ++t) {
                sum += v[t][h / (HEADS / KV)][c];
                /* a sum of integers is exact; the division by t + 1 is two roundings */
                if (fabs(out[t][h][c] - sum / (t + 1)) > fabs(sum) / (t + 1) * 0x1p-22) bad++;
            }
        }
    check(bad == 0, "means of the values");

    /* one token of the same sequence, without offsets: the mean of all */
    check(gq_kv4_attn(&cache, d_q, HEADS * HD, HEADS, 1, NULL, d_len, 1, TOK, 0.f, 1, 0, d_out, HEADS * HD, ws, need, NULL) == GQ_OK,
          "gq_kv4_attn of one token");
    static float one[HEADS][HD];
    hip(hipMemcpy(one, d_out, sizeof one, hipMemcpyDeviceToHost), "copy of the token");
    bad = 0;
    for (int h = 0; h < HEADS; ++h)
        for (int c = 0; c < HD; ++c)
            if (fabs(one[h][c] - out[TOK - 1][h][c]) > fabs(out[TOK - 1][h][c]) * 0x1p-21) bad++;
    check(bad == 0, "the last token alone");

    /* refusals */
    check(gq_kv4_attn(&cache, d_q, HEADS * HD, 5, TOK, d_start, d_len, TOK, 3 * PAGE, 0.f, 1, 0, d_out, HEADS * HD, ws, need,
                      NULL) == GQ_ERR_SHAPE, "heads that are no multiple");
    check(gq_kv4_read(&cache, TOK, d_start, d_len, d_K, d_K, NULL) == GQ_ERR_OVERLAP, "K and V in one place");
    check(gq_kv4_append(NULL, d_k, KV * HD, d_v, KV * HD, TOK, d_start, d_len, NULL, NULL, NULL, 0, 0, NULL, NULL, 0, 0.f,
                        NULL) == GQ_ERR_NULL, "no cache");
    hip(hipStreamDestroy(s), "hipStreamDestroy");
    if (failures) return 1;
    printf("c client ok\n");
    return 0;
}
