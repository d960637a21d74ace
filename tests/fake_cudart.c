/* A stand-in for the CUDA runtime, preloaded in front of it, so that the
 * library's host code runs without a GPU: device memory is made-up addresses
 * that nothing dereferences, launches are written to a log in the order in
 * which they come.  One line per event: "<thread> <event> <details>". */
#define _GNU_SOURCE
#include <dlfcn.h>
#include <pthread.h>
#include <stdio.h>
#include <string.h>
#include <unistd.h>

enum { SUCCESS = 0, NO_MEMORY = 2 };

static pthread_mutex_t mu = PTHREAD_MUTEX_INITIALIZER;
static char text[1 << 20];
static size_t used;
static size_t next_address = 0x700000000000ull;
static size_t limit = (size_t)1 << 38;
static int last_error, device, status_word, launch_us, registers = 0, sms = 152;
static struct { const void *fun; char name[160]; } kernels[1024];
static int n_kernels;
static _Thread_local int thread_id;
static int threads;

static void note(const char *event, const char *detail, size_t a, size_t b) {
    pthread_mutex_lock(&mu);
    if (!thread_id) thread_id = ++threads;
    if (used < sizeof text - 512)
        used += (size_t)snprintf(text + used, 512, "%d %s %.300s %zx %zx\n", thread_id, event, detail, a, b);
    pthread_mutex_unlock(&mu);
}
static const char *name_of(const void *fun) {
    for (int i = 0; i < n_kernels; ++i)
        if (kernels[i].fun == fun) return kernels[i].name;
    return "?";
}

/* What a test sets and reads. */
void fake_set(size_t most_bytes, int status, int us) { limit = most_bytes, status_word = status, launch_us = us; }
void fake_registers(int n) { registers = n; }
void fake_multiprocessors(int n) { sms = n; }  /* before the first call */
int fake_last_error(void) { return last_error; }
/* Names of the library's kernels, one per line. */
size_t fake_kernels(char *out, size_t n) {
    size_t m = 0;
    for (int i = 0; i < n_kernels && m + 161 < n; ++i) m += (size_t)snprintf(out + m, n - m, "%s\n", kernels[i].name);
    return m;
}
size_t fake_log(char *out, size_t n) {
    pthread_mutex_lock(&mu);
    size_t m = used < n ? used : n;
    memcpy(out, text, m);
    used = 0;
    pthread_mutex_unlock(&mu);
    return m;
}

void __cudaRegisterFunction(void **fat, const char *host, char *dev, const char *name, int limit_, void *t, void *b,
                            void *bd, void *gd, int *w) {
    (void)dev, (void)fat, (void)limit_, (void)t, (void)b, (void)bd, (void)gd, (void)w;
    if (n_kernels < 1024) {
        kernels[n_kernels].fun = host;
        snprintf(kernels[n_kernels++].name, sizeof kernels[0].name, "%s", name);
    }
}
void **__cudaRegisterFatBinary(void *p) { (void)p; static void *h; return &h; }
void __cudaRegisterFatBinaryEnd(void **h) { (void)h; }
void __cudaUnregisterFatBinary(void **h) { (void)h; }
void __cudaRegisterVar(void **f, char *h, char *a, const char *n, int e, size_t s, int c, int g) {
    (void)f, (void)h, (void)a, (void)n, (void)e, (void)s, (void)c, (void)g;
}

int cudaGetDevice(int *d) { *d = device; return SUCCESS; }
int cudaDeviceGetAttribute(int *v, int attr, int d) {
    (void)d;
    *v = attr == 16 ? sms : 232448;  /* multiprocessors; opt-in shared memory */
    return SUCCESS;
}
int cudaMalloc(void **p, size_t n) {
    if (n > limit) {
        note("malloc", "refused", 0, n);
        return last_error = NO_MEMORY;
    }
    pthread_mutex_lock(&mu);
    *p = (void *)next_address;
    next_address += (n + 0xfffff) & ~(size_t)0xfffff;
    pthread_mutex_unlock(&mu);
    note("malloc", "ok", (size_t)*p, n);
    return SUCCESS;
}
int cudaFree(void *p) { note("free", "", (size_t)p, 0); return SUCCESS; }
int cudaGetLastError(void) { int e = last_error; last_error = 0; return e; }
const char *cudaGetErrorString(int e) { return e == NO_MEMORY ? "out of memory" : "no error"; }
int cudaDeviceSynchronize(void) { note("device-sync", "", 0, 0); return SUCCESS; }
int cudaStreamSynchronize(void *s) { note("stream-sync", "", (size_t)s, 0); return SUCCESS; }
int cudaMemcpy(void *dst, const void *src, size_t n, int kind) {
    (void)kind;
    note("memcpy", "", (size_t)src, n);
    if (n == sizeof status_word) memcpy(dst, &status_word, n);
    return SUCCESS;
}
int cudaMemset(void *p, int v, size_t n) { (void)v; note("memset", "", (size_t)p, n); return SUCCESS; }
int cudaMemsetAsync(void *p, int v, size_t n, void *s) { (void)v, (void)s; note("memset-async", "", (size_t)p, n); return SUCCESS; }
int cudaMemset2DAsync(void *p, size_t ld, int v, size_t w, size_t h, void *s) {
    (void)ld, (void)v, (void)w, (void)h, (void)s;
    note("memset2d", "", (size_t)p, w);
    return SUCCESS;
}
int cudaFuncSetAttribute(const void *f, int a, int v) { (void)f, (void)a, (void)v; return SUCCESS; }
int cudaFuncGetAttributes(void *attr, const void *f) {
    /* numRegs is the fourth word after three size_t */
    const char *n = name_of(f);
    memset(attr, 0, 64);
    const int dual = strstr(n, "f8_wide_kernelILi1ELb1E") || strstr(n, "f8_wide_kernelILi2ELb1E");
    ((int *)((size_t *)attr + 3))[1] = registers ? registers : dual ? 96 : 168;
    return SUCCESS;
}
int cudaOccupancyMaxActiveClusters(int *n, const void *f, const void *cfg) { (void)f, (void)cfg; *n = 76; return SUCCESS; }
int cudaGetSymbolAddress(void **p, const void *s) { (void)s; *p = (void *)0x600000000000ull; return SUCCESS; }
static int encode_any(void) { return 0; }
int cudaGetDriverEntryPointByVersion(const char *s, void **p, unsigned v, unsigned long long f, int *q) {
    (void)s, (void)v, (void)f;
    *p = (void *)encode_any;
    if (q) *q = 0;
    return SUCCESS;
}

/* cudaLaunchConfig_t: two dim3, a size_t, the stream */
int cudaLaunchKernelExC(const void *cfg, const void *f, void **args) {
    (void)args;
    note("launch", name_of(f), *(const size_t *)((const char *)cfg + 32), *(const unsigned *)cfg);
    if (launch_us) usleep((unsigned)launch_us);
    return SUCCESS;
}
static _Thread_local struct { unsigned g[3], b[3]; size_t smem; void *st; } pushed;
unsigned __cudaPushCallConfiguration(unsigned long long gxy, unsigned gz, unsigned long long bxy, unsigned bz, size_t smem,
                                     void *st) {
    (void)gxy, (void)gz, (void)bxy, (void)bz;
    pushed.smem = smem, pushed.st = st;
    return 0;
}
int __cudaPopCallConfiguration(void *g, void *b, size_t *smem, void *st) {
    memset(g, 0, 12), memset(b, 0, 12);
    *smem = pushed.smem, *(void **)st = pushed.st;
    return SUCCESS;
}
int __cudaGetKernel(void **k, const void *f) { *k = (void *)f; return SUCCESS; }
int __cudaLaunchKernel(void *k, unsigned long long gxy, unsigned gz, unsigned long long bxy, unsigned bz, void **args,
                       size_t smem, void *st) {
    (void)gxy, (void)gz, (void)bxy, (void)bz, (void)args, (void)smem;
    note("launch", name_of(k), (size_t)st, 0);
    if (launch_us) usleep((unsigned)launch_us);
    return SUCCESS;
}
