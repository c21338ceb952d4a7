/*
 * Host sanitizer driver for the entry points of cached keys and values and of beam
 * selection: tests/test_sanitizers_generation.py builds their argument checks and
 * workspace layouts with AddressSanitizer and UndefinedBehaviorSanitizer and links
 * this to them. Every member in turn, and then several at random, takes the values at
 * the edges of its type and of the documented limits. No call may launch: a pointer
 * that the call needs is always NULL. Any sanitizer report, or a status of success
 * from a call that lacks one, fails the run.
 */
#include <limits.h>
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "dws_scan.h"

static int g_bad = 0;
static uint64_t g_state = 2468;

static uint64_t draw(void)
{
    g_state = g_state * 6364136223846793005ull + 1442695040888963407ull;
    return g_state >> 33;
}

static const long long kWide[] = {LLONG_MIN, LLONG_MIN + 1, -(1ll << 40), -1, 0, 1, 2, 7, 16, 63, 64, 65, 1000, 65535, 65536,
                                  (1 << 24) - 1, 1 << 24, (1 << 24) + 1, INT_MAX - 4096, INT_MAX, 1ll << 31, (1ll << 32) - 1,
                                  (1ll << 40) - 1, 1ll << 40, (1ll << 40) + 1, 1ll << 50, 1ll << 62, LLONG_MAX - 1, LLONG_MAX};
static const int kNarrow[] = {INT_MIN, -1, 0, 1, 2, 3, 5, 7, 31, 32, 33, 63, 64, 65, 128, 255, 256, 257, 65535, 65536, INT_MAX};
#define WIDE (sizeof kWide / sizeof kWide[0])
#define NARROW (sizeof kNarrow / sizeof kNarrow[0])

static void expect(int right, const char* what)
{
    if (right) return;
    printf("unexpected status: %s\n", what);
    g_bad = 1;
}

static void* at(uint64_t i) { return (void*)(uintptr_t)(0x100000ull + 0x10000000ull * i); }

static dws_rows rows(int i, long long ts, long long hs)
{
    dws_rows r = {at((uint64_t)i), ts, hs};
    return r;
}

/* The members of a cache and a call's tokens that are numbers. */
static void change_cache(dws_kv_cache* c, dws_page_seqs* s, uint64_t which, uint64_t value)
{
    long long* wide[] = {&c->keys.page_stride, &c->keys.token_stride, &c->keys.head_stride, &c->values.page_stride,
                         &c->values.token_stride, &c->values.head_stride, &c->n_pages, &c->n_rows, &c->max_pages,
                         &c->page_tokens, &s->tokens, &s->n};
    int* narrow[] = {&c->heads, &c->dim_k, &c->dim_v, &c->dtype};
    which %= 16;
    if (which < 12)
        *wide[which] = kWide[value % WIDE];
    else
        *narrow[which - 12] = kNarrow[value % NARROW];
}

static dws_kv_cache cache(void)
{
    dws_kv_cache c;
    memset(&c, 0, sizeof c);
    c.keys.data = at(1);
    c.values.data = at(2);
    c.keys.page_stride = c.values.page_stride = 16 * 4 * 64;
    c.keys.token_stride = c.values.token_stride = 4 * 64;
    c.keys.head_stride = c.values.head_stride = 64;
    c.d_table = (const int*)at(3);
    c.d_lengths = (const int*)at(4);
    c.n_pages = 100;
    c.n_rows = 10;
    c.max_pages = 20;
    c.page_tokens = 16;
    c.heads = 4;
    c.dim_k = c.dim_v = 64;
    c.dtype = DWS_BFLOAT16;
    return c;
}

static void append_calls(void)
{
    expect(dws_pages_append(NULL, NULL) != DWS_OK, "append of nothing");
    for (int r = 0; r < 40000; ++r) {
        dws_pages_append_args a;
        memset(&a, 0, sizeof a);
        a.cache = cache();
        a.seqs.tokens = a.seqs.n = 8;
        a.pairs = 32;
        a.d_freqs = (const float*)at(5);
        a.heads_q = 8;
        a.k = rows(6, 256, 64);
        a.v = rows(7, 256, 64);
        a.q = rows(8, 512, 64);
        a.q_out = rows(9, 512, 64);
        const int changes = r < 16 * (int)WIDE ? 1 : 1 + (int)(draw() % 4);
        for (int k = 0; k < changes; ++k) {
            const uint64_t which = r < 16 * (int)WIDE ? (uint64_t)r / WIDE : draw() % 24;
            const uint64_t value = r < 16 * (int)WIDE ? (uint64_t)r : draw();
            long long* wide[] = {&a.k.token_stride, &a.k.head_stride, &a.v.token_stride, &a.v.head_stride, &a.q.token_stride, &a.q_out.head_stride};
            if (which < 16)
                change_cache(&a.cache, &a.seqs, which, value);
            else if (which < 22)
                *wide[which - 16] = kWide[value % WIDE];
            else if (which == 22)
                a.pairs = kNarrow[value % NARROW];
            else
                a.heads_q = kNarrow[value % NARROW];
        }
        a.cache.values.data = NULL;
        expect(dws_pages_append(&a, NULL) != DWS_OK, "append");
    }
}

static void attention_calls(void)
{
    size_t bytes = 0;
    expect(dws_pages_attention(NULL, NULL) != DWS_OK, "attention of nothing");
    expect(dws_pages_attention_workspace(NULL, &bytes) != DWS_OK, "workspace of nothing");
    for (int r = 0; r < 40000; ++r) {
        dws_pages_attention_args a;
        memset(&a, 0, sizeof a);
        a.cache = cache();
        a.seqs.tokens = a.seqs.n = 8;
        a.heads_q = 16;
        a.scale = r % 7 == 3 ? (float)INFINITY : .125f;
        a.n_groups = r % 2 ? 3 : 0;
        a.d_groups = (const long long*)at(5);
        a.d_shared = (const int*)at(6);
        a.q = rows(8, 1024, 64);
        a.out = rows(9, 1024, 64);
        a.d_lse = (float*)at(10);
        a.workspace_bytes = SIZE_MAX;
        const int changes = r < 16 * (int)WIDE ? 1 : 1 + (int)(draw() % 4);
        for (int k = 0; k < changes; ++k) {
            const uint64_t which = r < 16 * (int)WIDE ? (uint64_t)r / WIDE : draw() % 21;
            const uint64_t value = r < 16 * (int)WIDE ? (uint64_t)r : draw();
            long long* wide[] = {&a.n_groups, &a.q.token_stride, &a.q.head_stride, &a.out.token_stride};
            if (which < 16)
                change_cache(&a.cache, &a.seqs, which, value);
            else if (which < 20)
                *wide[which - 16] = kWide[value % WIDE];
            else
                a.heads_q = kNarrow[value % NARROW];
        }
        bytes = 0;
        if (dws_pages_attention_workspace(&a, &bytes) == DWS_OK)
            expect(bytes > 0 && bytes < (size_t)1 << 60, "bytes of workspace");
        expect(dws_pages_attention_workspace(&a, NULL) != DWS_OK, "workspace without a place for its size");
        a.d_workspace = NULL;
        expect(dws_pages_attention(&a, NULL) != DWS_OK, "attention");
    }
}

static void beam_calls(void)
{
    size_t bytes = 0;
    expect(dws_beam_select(NULL, NULL) != DWS_OK, "beams of nothing");
    expect(dws_beam_select_workspace(NULL, &bytes) != DWS_OK, "workspace of nothing");
    for (int r = 0; r < 40000; ++r) {
        dws_beam_args a;
        memset(&a, 0, sizeof a);
        a.d_logits = at(1);
        a.batch = 3;
        a.beams = a.k = 4;
        a.vocab = 1000;
        a.beam_stride = 1000;
        a.batch_stride = 4000;
        a.dtype = DWS_FLOAT32;
        a.d_scores = (const float*)at(2);
        a.d_finished = r % 2 ? (const unsigned char*)at(3) : NULL;
        a.d_rows = r % 3 ? (const int*)at(4) : NULL;
        a.d_out_scores = (float*)at(5);
        a.d_parents = (int*)at(6);
        a.d_tokens = (int*)at(7);
        a.d_out_rows = (int*)at(8);
        a.d_src = (int*)at(9);
        a.d_dst = (int*)at(10);
        a.workspace_bytes = SIZE_MAX;
        long long* wide[] = {&a.batch, &a.beams, &a.vocab, &a.batch_stride, &a.beam_stride, &a.end_token};
        int* narrow[] = {&a.dtype, &a.k};
        for (int k = 1 + (int)(draw() % 3); k > 0; --k) {
            const uint64_t which = draw() % 8;
            if (which < 6)
                *wide[which] = kWide[draw() % WIDE];
            else
                *narrow[which - 6] = kNarrow[draw() % NARROW];
        }
        bytes = 0;
        if (dws_beam_select_workspace(&a, &bytes) == DWS_OK) expect(bytes < (size_t)1 << 50, "bytes of workspace");
        expect(dws_beam_select_workspace(&a, NULL) != DWS_OK, "workspace without a place for its size");
        expect(dws_beam_select(&a, NULL) != DWS_OK || a.batch == 0, "beams");
    }
}

int main(void)
{
    append_calls();
    attention_calls();
    beam_calls();
    if (!g_bad) printf("generation driver: ok\n");
    return g_bad;
}
