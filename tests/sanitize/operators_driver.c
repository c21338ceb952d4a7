/*
 * Host sanitizer driver for the entry points of the delta rule and the pages:
 * tests/test_sanitizers_operators.py builds their argument checks and workspace
 * layout with AddressSanitizer and UndefinedBehaviorSanitizer and links this to
 * them. Every member in turn, and then all of them at random, takes the values
 * at the edges of its type and of the documented limits. No call may launch: a
 * pointer that the call needs is always NULL. Any sanitizer report, or a status
 * of success from a call that lacks one, fails the run.
 */
#include <limits.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "dws_scan.h"

static int g_bad = 0;
static uint64_t g_state = 12345;

static uint64_t draw(void)
{
    g_state = g_state * 6364136223846793005ull + 1442695040888963407ull;
    return g_state >> 33;
}

static const long long kWide[] = {LLONG_MIN, LLONG_MIN + 1, -(1ll << 40), -1, 0, 1, 2, 63, 64, 65, 255, 256, 257, 4095, 65535,
                                  65536, (1 << 22) - 1, 1 << 22, (1 << 24) - 1, 1 << 24, (1 << 24) + 1, INT_MAX, 1ll << 31,
                                  (1ll << 32) - 1, 1ll << 40, (1ll << 40) + 1, 1ll << 50, 1ll << 62, LLONG_MAX - 1, LLONG_MAX};
static const int kNarrow[] = {INT_MIN, -1, 0, 1, 2, 3, 5, 6, 7, 16, 64, 128, 255, 256, 257, 65535, 65536, INT_MAX};
#define WIDE (sizeof kWide / sizeof kWide[0])
#define NARROW (sizeof kNarrow / sizeof kNarrow[0])

static void* at(uint64_t i) { return (void*)(uintptr_t)(0x100000ull + 0x1000000ull * i); }

static dws_rows rows(int i, long long ts, long long hs)
{
    dws_rows r = {at((uint64_t)i), ts, hs};
    return r;
}

static dws_delta_rule_args arguments(void)
{
    dws_delta_rule_args a;
    memset(&a, 0, sizeof a);
    a.tokens = 128;
    a.n_seqs = 2;
    a.heads_qk = 2;
    a.heads_v = 4;
    a.dim_k = a.dim_v = 64;
    a.dtype = DWS_BFLOAT16;
    a.g_dtype = DWS_FLOAT32;
    a.beta_dtype = DWS_FLOAT16;
    a.scale = 1.f;
    a.q = rows(1, 128, 64);
    a.k = rows(2, 128, 64);
    a.v = rows(3, 256, 64);
    a.g = rows(4, 4, 1);
    a.beta = rows(5, 4, 1);
    a.out = rows(6, 256, 64);
    a.d_slots = 0;
    a.n_states = 0;
    a.out_grad = rows(7, 256, 64);
    a.q_grad = rows(8, 128, 64);
    a.k_grad = rows(9, 128, 64);
    a.v_grad = rows(10, 256, 64);
    a.g_grad = rows(11, 4, 1);
    a.beta_grad = rows(12, 4, 1);
    a.workspace_bytes = SIZE_MAX;       /* and d_workspace NULL */
    return a;
}

static void expect(int refused, const char* what)
{
    if (!refused) {
        fprintf(stderr, "FAIL: %s succeeded\n", what);
        g_bad = 1;
    }
}

static void delta(const dws_delta_rule_args* a)
{
    size_t bytes = 0;
    for (int backward = 0; backward < 2; ++backward)
        if (dws_delta_rule_workspace(a, backward, &bytes) == DWS_OK) expect(bytes > 0, "a workspace of no bytes");
    expect(dws_delta_rule(a, NULL) != DWS_OK, "dws_delta_rule without a workspace");
    expect(dws_delta_rule_backward(a, NULL) != DWS_OK, "dws_delta_rule_backward without a workspace");
    expect(dws_delta_rule_step(a, NULL) != DWS_OK, "dws_delta_rule_step without a state");
}

static void delta_rule(void)
{
    dws_delta_rule_args a = arguments();
    long long* wide[] = {&a.tokens, &a.n_seqs, &a.n_states, &a.q.token_stride, &a.q.head_stride, &a.v.token_stride, &a.g.token_stride,
                         &a.out.token_stride, &a.out.head_stride, &a.out_grad.head_stride, &a.q_grad.token_stride,
                         &a.beta_grad.head_stride};
    int* narrow[] = {&a.heads_qk, &a.heads_v, &a.dim_k, &a.dim_v, &a.dtype, &a.g_dtype, &a.beta_dtype};
    const size_t nw = sizeof wide / sizeof wide[0], nn = sizeof narrow / sizeof narrow[0];
    delta(&a);
    for (size_t i = 0; i < nw; ++i)
        for (size_t j = 0; j < WIDE; ++j) {
            a = arguments();
            *wide[i] = kWide[j];
            delta(&a);
        }
    for (size_t i = 0; i < nn; ++i)
        for (size_t j = 0; j < NARROW; ++j) {
            a = arguments();
            *narrow[i] = kNarrow[j];
            delta(&a);
        }
    for (int r = 0; r < 20000; ++r) {
        a = arguments();
        for (int k = (int)(draw() % 5); k >= 0; --k) {
            if (draw() % 2)
                *wide[draw() % nw] = kWide[draw() % WIDE];
            else
                *narrow[draw() % nn] = kNarrow[draw() % NARROW];
        }
        if (draw() % 3 == 0) a.d_offsets = (const long long*)at(20);
        if (draw() % 3 == 0) a.d_slots = (const int*)at(21);
        if (draw() % 3 == 0) a.d_initial_state = (const float*)at(22);
        if (draw() % 4 == 0) a.v.data = (char*)a.v.data + 1 + draw() % 8;
        if (draw() % 8 == 0) a.out.data = (void*)(uintptr_t)(UINTPTR_MAX - draw() % 4096);
        delta(&a);
    }
    delta(NULL);
}

static void pages(const dws_page_cache* c, long long n)
{
    size_t bytes = 0;
    if (dws_pages_workspace(c, n, &bytes) == DWS_OK) expect(bytes > 0, "a workspace of no bytes");
    const int* in = (const int*)at(30);
    int* out = (int*)at(40);
    long long* one = (long long*)at(50);
    expect(dws_pages_grow(c, in, (const int*)at(31), n, out, NULL, SIZE_MAX, NULL) != DWS_OK, "grow");
    expect(dws_pages_fork(c, in, (const int*)at(31), n, out, (int*)at(41), (int*)at(42), one, NULL, SIZE_MAX, NULL) != DWS_OK, "fork");
    expect(dws_pages_free(c, in, n, one, NULL, SIZE_MAX, NULL) != DWS_OK, "free");
    expect(dws_pages_compact(c, out, (int*)at(41), (int*)at(42), one, (long long*)at(51), NULL, SIZE_MAX, NULL) != DWS_OK, "compact");
}

static void page_calls(void)
{
    for (int r = 0; r < 20000; ++r) {
        dws_page_cache c = {(int*)at(1), 100, (int*)at(2), 10, 20, (int*)at(3), 16};
        long long n = 5;
        long long* wide[] = {&c.n_pages, &c.n_rows, &c.max_pages, &c.page_tokens, &n};
        if (r < (int)(5 * WIDE))
            *wide[r / WIDE] = kWide[r % WIDE];
        else
            for (int k = (int)(draw() % 4); k >= 0; --k) *wide[draw() % 5] = kWide[draw() % WIDE];
        pages(&c, n);
        /* copies without a pool, or with nothing to copy */
        long long v[5] = {100, 4096, 2, 1 << 20, 7};
        for (int k = (int)(draw() % 5); k > 0; --k) v[draw() % 5] = kWide[draw() % WIDE];
        const dws_status st = dws_pages_copy(NULL, v[0], v[1], v[2], v[3], (const int*)at(30), (const int*)at(31), v[4], NULL, NULL);
        expect(st != DWS_OK || v[0] == 0 || v[1] == 0 || v[2] == 0 || v[4] == 0, "copy");
    }
    pages(NULL, 1);
}

int main(void)
{
    delta_rule();
    page_calls();
    if (!g_bad) printf("operators driver: ok\n");
    return g_bad;
}
