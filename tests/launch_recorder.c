/* Stands in for the HIP runtime's launch functions, so that a process without a GPU can ask
 * libzx.so what it would launch.  Loaded with RTLD_GLOBAL before the library, whose references
 * then bind here; nothing reaches a device. */
#include <stddef.h>
#include <stdint.h>
#include <string.h>

typedef struct { uint32_t x, y, z; } dim3;
typedef struct { char name[256]; dim3 grid, block; unsigned char arg[512]; } record;

enum { MOST = 4096, KERNELS = 1024 };
record zr_launches[MOST];
int zr_count;
static struct { const void *f; const char *name; } kernels[KERNELS];
static int n_kernels;
static dim3 c_grid, c_block;
static size_t c_lds;
static void *c_stream;

void **__hipRegisterFatBinary(const void *data) { static void *one; (void)data; return &one; }
void __hipUnregisterFatBinary(void **m) { (void)m; }
void __hipRegisterVar(void) {}
void __hipRegisterFunction(void **m, const void *f, char *dev, const char *name, unsigned n, void *a, void *b, void *c, void *d, int *w)
{
    (void)m; (void)dev; (void)n; (void)a; (void)b; (void)c; (void)d; (void)w;
    if (n_kernels < KERNELS) {
        kernels[n_kernels].f = f;
        kernels[n_kernels++].name = name;
    }
}
int __hipPushCallConfiguration(dim3 g, dim3 b, size_t lds, void *s) { c_grid = g; c_block = b; c_lds = lds; c_stream = s; return 0; }
int __hipPopCallConfiguration(dim3 *g, dim3 *b, size_t *lds, void **s) { *g = c_grid; *b = c_block; *lds = c_lds; *s = c_stream; return 0; }
int hipGetLastError(void) { return 0; }
/* `zr_bytes`: size of the kernels' only argument, a struct */
size_t zr_bytes;
int hipLaunchKernel(const void *f, dim3 g, dim3 b, void **args, size_t lds, void *s)
{
    (void)lds; (void)s;
    if (zr_count == MOST) return 1;
    record *r = &zr_launches[zr_count++];
    r->name[0] = 0;
    for (int i = 0; i < n_kernels; ++i)
        if (kernels[i].f == f) strncpy(r->name, kernels[i].name, sizeof r->name - 1);
    r->grid = g;
    r->block = b;
    memcpy(r->arg, args[0], zr_bytes < sizeof r->arg ? zr_bytes : sizeof r->arg);
    return 0;
}
